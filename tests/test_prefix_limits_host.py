"""Host-side checks at the limits of what the operators around a prefix cache allow (no GPU: no call here reaches a kernel)."""
import os
import shutil
import subprocess

import pytest

from test_ops_host import NULL, _call, _i, _z, gdn  # noqa: F401
from test_prefix_host import _sample, _shared


def test_a_prefix_without_cached_tokens_needs_its_pages(gdn):  # noqa: F811
    # no token is cached yet, but prefix_len may be up to max_prefix_len: its pages would be read
    for i in (1, 2, 3):
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=32, max_own_len=0), 10, {i: None}, ws_bytes=255) == NULL, i
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=1), 10, {i: None}, ws_bytes=255) == NULL, i


def test_bounds_of_a_prefix_beyond_every_kv_len(gdn):  # noqa: F811
    q, kc, table = _z(2, 8, 128), _z(10, 16, 2, 128), _i(1, 2, 3, 4, 5, 6).view(2, 3)

    def bounds(**kw):
        d = gdn.make_shared_desc(q, kc, table, 2, 1, **kw)
        return d.cache.max_kv_len, d.max_prefix_len, d.max_own_len

    assert bounds() == (48, 48, 48) and bounds(max_kv_len=35) == (35, 35, 35)
    assert bounds(max_kv_len=35, max_prefix_len=40) == (35, 40, 35)
    assert bounds(max_kv_len=35, max_prefix_len=100, max_own_len=40) == (35, 48, 35)      # as much as a table's row holds
    assert bounds(max_kv_len=0, max_prefix_len=40, max_own_len=0) == (0, 40, 0)
    assert bounds(max_kv_len=1 << 30, max_prefix_len=1 << 30, max_own_len=7) == (48, 48, 7)


def test_sample_workspace_serves_fewer_rows(gdn):  # noqa: F811
    for dtype in (0, 1):
        for vocab in (1, 100, 2049, 8192, 8193, 32000, 49999, 65536, 65537, 131072, 1 << 24):
            need = [gdn.gdn_sample_workspace_bytes(_sample(gdn, rows=r, vocab=vocab, stride=vocab, dtype=dtype)) for r in range(0, 500)]
            assert need == sorted(need), (dtype, vocab)


PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "gdn_plan.h"
using namespace gdn;
int main()
{
    // bf16 probabilities are as fine as without groups: by the rows of a sequence, whatever form a prefix takes
    for (int64_t t : {1LL, 64LL, 65LL, 1501LL}) for (int n : {1, 16, 64, 100}) for (int g : {1, 4, 100}) for (int h : {1, 8}) for (int rep : {1, 8, 32})
        for (int d : {64, 128, 256}) for (int pre : {0, 700, 31744}) for (int own : {0, 40, 5000}) {
            const SharedPlan p = shared_plan(t, n, g, h * rep, h, d, pre, own, 1);
            if (p.fine != attn_plan(t, n, h * rep, h, d, pre + own, 1).decode) return 1;
            if (own > 0 && p.own.decode != p.fine) return 2;
        }
    // what the test on the GPU of that relies on
    const int at[][6] = {%s};
    for (auto &c : at) {
        const SharedPlan p = shared_plan(c[3], c[3], c[4], c[0] * c[1], c[0], c[2], 31744, 700, 1);
        if (p.prefix.decode || p.prefix.rows != c[5] || !p.fine) {
            printf("d %%d, %%d requests: decode %%d, rows %%d\n", c[2], c[3], p.prefix.decode, p.prefix.rows);
            return 3;
        }
    }
    puts("plans: ok");
    return 0;
}
"""


def test_plans_keep_the_precision_of_few_rows(tmp_path):
    from test_gpu_prefix_limits import FINE
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "plans.cpp", str(tmp_path / "plans")
    src.write_text(PROGRAM % ", ".join("{%d, %d, %d, %d, %d, %d}" % (*c, 128 if c[3] == 32 else 256) for c in FINE))
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", os.path.join(root, "gated_deltanet_state_gdn_amd", "csrc"), str(src), "-o", exe])
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, (p.returncode, p.stdout)
