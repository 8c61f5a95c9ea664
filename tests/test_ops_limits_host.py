"""Host-side limits of the suffix and decode operators: sizes whose products leave 64 bits, grids that
one launch does not hold.  No call here reaches a kernel.  Run once more against the library whose
argument validation is built with ASan and UBSan."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_ops_host import N, P, SHAPE, _call, _fill, _paged, gdn  # noqa: F401 (gdn: the fixture)

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


def test_grids_beyond_one_launch(gdn):  # noqa: F811
    """A grid holds fewer than 2^32 threads, whatever a workgroup has: refused in front of the call's first
    launch (without a GPU a launch answers otherwise)."""
    def ssm(**kw):
        return _fill(gdn._lib.GdnSsmDesc, dict(n_seqs=1, n_slots=1, h_qk=1, h_v=1, d_k=64, d_v=128, dtype=1, softplus=1,
                                               total_tokens=1, total_out_tokens=1, b_stride=64, c_stride=64), kw)

    rows, seqs = 268435455, 4000000                                     # workgroups of 512 threads over 256 rows of 8 heads
    d = _paged(gdn, n_seqs=seqs, h_q=8, h_kv=1, d=64, max_kv_len=64, total_tokens=rows, q_stride=512, o_stride=512, head_stride=64)
    assert (rows * 8 // 256 + seqs) < 1 << 24 and _call(gdn, "gdn_paged_attn", d, 8) == SHAPE
    d = ssm(n_seqs=1 << 20, h_v=12, total_tokens=1 << 20, total_out_tokens=1 << 20, x_stride=1536, y_stride=1536, dt_stride=12)
    assert _call(gdn, "gdn_ssm_scan", d, 13) == SHAPE                   # of 512 threads over 128 columns; cu_out asked for
    big = 0x7fffffff
    d = ssm(n_seqs=big, n_slots=big, h_v=64, total_tokens=big, total_out_tokens=big, x_stride=8192, y_stride=8192, dt_stride=64)
    assert _call(gdn, "gdn_ssm_step", d, 10) == SHAPE
    d = _fill(gdn._lib.GdnDesc, dict(n_seqs=big, h_qk=big, h_v=big, d_k=128, d_v=128, qkv_dtype=1, o_dtype=1, scale=1.0,
                                     total_tokens=big, total_out_tokens=big), {})
    assert gdn.load().gdn_step(ctypes.byref(d), *[P] * 6, big, P, P, P, 256, None) == SHAPE
    d = _fill(gdn._lib.GdnConvDesc, dict(n_seqs=big, n_slots=big, channels=512, width=4, dtype=1, silu=1, total_tokens=big,
                                         x_stride=512, y_stride=512), {})
    assert _call(gdn, "gdn_conv_step", d, 6) == SHAPE and _call(gdn, "gdn_conv", d, 7) == SHAPE
    d = _paged(gdn, n_seqs=1, h_q=8, total_tokens=1 << 27)
    assert _call(gdn, "gdn_qk_norm_rope", d, 13) == SHAPE
