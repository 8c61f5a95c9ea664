"""Host-side checks of the operators around a prefix cache (no GPU: no call here reaches a kernel)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

from test_ops_host import (ALIGN, BIG, DTYPE, NULL, P, PM, SHAPE, UNSUPPORTED, WORKSPACE, _call, _fill, _i, _paged,  # noqa: F401
                           _refused, _z, gdn)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ODD = ctypes.c_void_p(0x100001)


def _shared(g, n_groups=1, max_prefix_len=32, max_own_len=48, **kw):
    return g._lib.GdnSharedDesc(cache=_paged(g, **kw), n_groups=n_groups, max_prefix_len=max_prefix_len, max_own_len=max_own_len)


def _extend(g, **kw):
    return _fill(g._lib.GdnExtendDesc, dict(n_seqs=3, page_size=16, max_pages=4, n_free=10, n_prefixes=2, max_prefix_pages=3,
                                            total_tokens=20), kw)


def _sample(g, **kw):
    return _fill(g._lib.GdnSampleDesc, dict(rows=3, vocab=1000, dtype=1, stride=1000), kw)


N = {"gdn_shared_attn": 10, "gdn_cache_extend": 13, "gdn_sample": 8}
MAKE = {"gdn_shared_attn": _shared, "gdn_cache_extend": _extend, "gdn_sample": _sample}
OPTIONAL = {"gdn_shared_attn": {9}, "gdn_cache_extend": {11, 12}, "gdn_sample": {2, 3, 4, 5, 7}}
NARROW = {"gdn_shared_attn": {3, 4, 5, 6, 7, 9}, "gdn_cache_extend": set(range(13)) - {11}, "gdn_sample": {1, 2, 3, 4, 5, 6, 7}}
DESC_ERRORS = [
    ("gdn_shared_attn", dict(n_groups=-1), SHAPE), ("gdn_shared_attn", dict(n_groups=0), SHAPE),
    ("gdn_shared_attn", dict(max_prefix_len=-1), SHAPE), ("gdn_shared_attn", dict(max_own_len=-1), SHAPE),
    ("gdn_shared_attn", dict(max_prefix_len=(1 << 30) + 1), SHAPE), ("gdn_shared_attn", dict(max_own_len=(1 << 30) + 1), SHAPE),
    ("gdn_shared_attn", dict(h_q=7), SHAPE), ("gdn_shared_attn", dict(d=96), UNSUPPORTED), ("gdn_shared_attn", dict(dtype=2), DTYPE),
    ("gdn_shared_attn", dict(scale=float("nan")), SHAPE), ("gdn_shared_attn", dict(q_stride=1020), ALIGN),
    ("gdn_shared_attn", dict(o_stride=1000), ALIGN), ("gdn_shared_attn", dict(token_stride=120), ALIGN),
    ("gdn_cache_extend", dict(n_seqs=-1), SHAPE), ("gdn_cache_extend", dict(page_size=0), SHAPE),
    ("gdn_cache_extend", dict(max_pages=-1), SHAPE), ("gdn_cache_extend", dict(n_free=-1), SHAPE),
    ("gdn_cache_extend", dict(n_prefixes=-1), SHAPE), ("gdn_cache_extend", dict(max_prefix_pages=-1), SHAPE),
    ("gdn_cache_extend", dict(total_tokens=-1), SHAPE), ("gdn_cache_extend", dict(total_tokens=1 << 31), SHAPE),
    ("gdn_sample", dict(rows=-1), SHAPE), ("gdn_sample", dict(vocab=0), SHAPE), ("gdn_sample", dict(vocab=(1 << 24) + 1, stride=1 << 25), SHAPE),
    ("gdn_sample", dict(stride=999), SHAPE), ("gdn_sample", dict(stride=1 << 40), SHAPE), ("gdn_sample", dict(dtype=2), DTYPE),
]


@pytest.mark.parametrize("name,change,code", DESC_ERRORS)
def test_descriptor_refusals(gdn, name, change, code):  # noqa: F811
    assert _call(gdn, name, MAKE[name](gdn, **change), N[name]) == code


@pytest.mark.parametrize("name", sorted(N))
def test_pointer_refusals(gdn, name):  # noqa: F811
    d = MAKE[name](gdn)
    for i in range(N[name]):
        if i not in OPTIONAL[name]:
            assert _call(gdn, name, d, N[name], {i: None}) == NULL, i
        assert _call(gdn, name, d, N[name], {i: ODD if i in NARROW[name] or name != "gdn_shared_attn" else PM}) == ALIGN, i
    assert _call(gdn, name, None, N[name]) == NULL
    assert _call(gdn, name, d, N[name], ws=None) == NULL
    assert _call(gdn, name, d, N[name], ws=PM) == ALIGN
    assert _call(gdn, name, d, N[name], ws_bytes=255) == WORKSPACE


def test_nothing_to_do_is_accepted(gdn):  # noqa: F811
    assert _call(gdn, "gdn_shared_attn", _shared(gdn, n_seqs=0, total_tokens=0, n_groups=0), 10) == 0
    assert _call(gdn, "gdn_shared_attn", _shared(gdn, total_tokens=0), 10) == 0
    assert _call(gdn, "gdn_sample", _sample(gdn, rows=0), 8, {0: None, 1: None, 6: None}) == 0


def test_prefixes_need_their_tables(gdn):  # noqa: F811
    for i in (5, 6, 7):
        assert _call(gdn, "gdn_cache_extend", _extend(gdn), 13, {i: None}) == NULL


def test_workspace_sizes(gdn):  # noqa: F811
    for name, d, need in (("gdn_shared_attn", _shared(gdn), gdn.gdn_shared_workspace_bytes(_shared(gdn))),
                          ("gdn_cache_extend", _extend(gdn), gdn.gdn_extend_workspace_bytes(3)),
                          ("gdn_sample", _sample(gdn), gdn.gdn_sample_workspace_bytes(_sample(gdn)))):
        assert need > 256 and _call(gdn, name, d, N[name], ws_bytes=need - 1) == WORKSPACE, name
    assert gdn.gdn_shared_workspace_bytes(_shared(gdn, d=80)) == 0 and gdn.gdn_sample_workspace_bytes(_sample(gdn, vocab=0)) == 0
    assert gdn.gdn_extend_workspace_bytes(-1) == 0
    r = random.Random(4)
    for _ in range(2000):
        n, total = r.choice([1, 2, 17, 300, 100000]), r.choice([0, 1, 5, 64, 1000, 70000, 1 << 24])
        h_kv, group, d = r.choice([1, 2, 8]), r.choice([1, 3, 8, 32]), r.choice([64, 128, 256])
        pre, own = (r.choice([0, 1, 63, 64, 257, 4095, 4096, 100001, 1 << 30]) for _ in range(2))
        if total * h_kv * group > 0x7fffffff:
            continue
        s = _shared(gdn, r.choice([1, n]), pre, own, n_seqs=n, total_tokens=total, h_q=h_kv * group, h_kv=h_kv, d=d, max_kv_len=1 << 30,
                    dtype=r.choice([0, 1]), token_stride=2048, head_stride=256, page_stride=32768)
        need, part = gdn.gdn_shared_workspace_bytes(s), total * h_kv * group * (d + 2) * 4
        assert 256 <= need <= 512 + part * (max(1, -(-pre // 32)) + max(1, -(-own // 32))), (n, total, h_kv, group, d, pre, own)
        rows, vocab = r.choice([1, 7, 300, 100000]), r.choice([1, 2047, 2048, 2049, 131072, 1 << 24])
        need = gdn.gdn_sample_workspace_bytes(_sample(gdn, rows=rows, vocab=vocab, stride=vocab))
        chunks = rows * (-(-vocab // 2048) + 1)
        assert rows * 2064 < need <= 1024 + chunks * 2064, (rows, vocab)


def test_python_refusals(gdn):  # noqa: F811
    f = torch.float32
    q, kc, table, cu, kv = _z(6, 8, 128), _z(10, 16, 2, 128), _i(1, 2, 3, 4).view(2, 2), _i(0, 2, 6), _i(20, 30)
    groups, pre = _i(0, 2), _i(16)
    at = gdn.gdn_shared_attn
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, groups, _i(16, 16))
    _refused(gdn, DTYPE, at, q, kc, kc, table, cu, kv, groups.long(), pre)
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, _i()[:0], pre)
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, groups, pre, max_prefix_len=-1)
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, groups, pre, max_own_len=1 << 31)
    _refused(gdn, DTYPE, at, q, kc.float(), kc.float(), table, cu, kv, groups, pre)
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, groups, pre, lse=_z(8, 6, dtype=f))
    _refused(gdn, NULL, at, q, kc, kc, table, cu, kv, None, pre)
    _refused(gdn, SHAPE, at, q, kc, kc, table, cu, kv, groups, pre)                     # on the CPU
    ext, new, free, one = gdn.gdn_cache_extend, _i(3, 4), _i(5, 6, 7), _i(0)
    _refused(gdn, SHAPE, ext, new, kv[:1], table, free, one, 16, 7)
    _refused(gdn, DTYPE, ext, new.long(), kv, table, free, one, 16, 7)
    _refused(gdn, SHAPE, ext, new, kv, table, free, _i(0, 0), 16, 7)
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 0, 7)
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 16, -1)
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 16, 7, prefix_of=_i(0, -1))
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 16, 7, prefix_of=_i(0, -1), prefix_table=_i(1, 2), prefix_len=_i(16))
    _refused(gdn, DTYPE, ext, new, kv, table, free, one, 16, 7, slots=torch.zeros(7, dtype=torch.int32))
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 16, 7, positions=_i(1, 2))
    _refused(gdn, ALIGN, ext, new, kv, torch.zeros(4, 2, dtype=torch.int32)[::2], free, one, 16, 7)
    _refused(gdn, SHAPE, ext, new, kv, table, free, one, 16, 7)
    x, u = _z(3, 100), _z(3, dtype=f)
    smp = gdn.gdn_sample
    _refused(gdn, DTYPE, smp, x.half(), u)
    _refused(gdn, DTYPE, smp, x, u.double())
    _refused(gdn, SHAPE, smp, x, u[:2])
    _refused(gdn, SHAPE, smp, x[0], u)
    _refused(gdn, ALIGN, smp, _z(100, 3).t(), u)
    _refused(gdn, DTYPE, smp, x, u, top_k=u)
    _refused(gdn, SHAPE, smp, x, u, temperature=_z(1, dtype=f))
    _refused(gdn, DTYPE, smp, x, u, token=torch.zeros(3, dtype=torch.int64))
    _refused(gdn, SHAPE, smp, x, u)
    with pytest.raises(gdn.GdnError):
        gdn.make_sample_desc(x[0])


PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "gdn_plan.h"
using namespace gdn;
static bool side(const AttnPlan &p, int64_t most)
{
    if (most == 0) return p.splits == 0;
    const bool rows = p.decode ? p.rows == 16 || p.rows == 32 : p.rows == 64 || p.rows == 128 || p.rows == 256;
    return rows && p.split_keys > 0 && p.splits > 0 && (int64_t)p.splits * p.split_keys >= most && (int64_t)(p.splits - 1) * p.split_keys < most;
}
int main()
{
    // both sides' splits cover their keys, the last one not in vain
    const int32_t ends[] = {0, 1, 31, 32, 33, 511, 512, 513, 4095, 4096, 100001, 1 << 30};
    for (int64_t t : {1LL, 2LL, 33LL, 64LL, 1501LL, 100000LL}) for (int n : {1, 2, 64, 1000}) for (int g : {1, 2, 64}) for (int h : {1, 2, 8})
        for (int rep : {1, 3, 8, 32}) for (int d : {64, 128, 256}) for (int bf16 : {0, 1}) for (int32_t pre : ends) for (int32_t own : ends) {
            const SharedPlan p = shared_plan(t, n, g, h * rep, h, d, pre, own, bf16);
            if (!side(p.prefix, pre) || !side(p.own, own)) {
                printf("%lld %d %d %d %d %d %d %d %d\n", (long long)t, n, g, h, rep, d, bf16, pre, own);
                return 1;
            }
        }
    for (int64_t r : {1LL, 5LL, 256LL, 100000LL}) for (int v : {1, 2047, 2048, 2049, 131072, 1 << 24})
        if (sample_chunk(r, v) != 2048 && sample_chunk(r, v) != 8192) return 2;
    puts("plans: ok");
    return 0;
}
"""


@pytest.mark.parametrize("san", [None, "address,undefined"])
def test_plans_of_all_sizes(tmp_path, san):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "plans.cpp", str(tmp_path / "plans")
    src.write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "gated_deltanet_state_gdn_amd", "csrc"), str(src), "-o", exe]
    subprocess.check_call(cmd + (["-fsanitize=" + san, "-fno-sanitize-recover=all"] if san else []))
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "ok" in p.stdout, p.stdout + p.stderr[-2000:]
