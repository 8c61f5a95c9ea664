"""Host-side checks of the suffix and decode operators (no GPU: no call here reaches a kernel).

The C entry points' argument errors, the Python binding's, and the index arithmetic the kernels
use for tiles of packed sequences and places in a paged cache, compiled for the host.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x100000)      # fake addresses: every call returns from host validation
PM = ctypes.c_void_p(0x100008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_state_gdn_amd as gdn
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built here")
    gdn.load()
    return gdn


def _fill(struct, base, kw):
    s = struct()
    for k, v in {**base, **kw}.items():
        setattr(s, k, v)
    return s


def _conv(gdn, **kw):
    return _fill(gdn._lib.GdnConvDesc, dict(n_seqs=2, n_slots=4, channels=64, width=4, dtype=1, silu=1,
                                            total_tokens=2, x_stride=64, y_stride=64), kw)


def _ssm(gdn, **kw):
    return _fill(gdn._lib.GdnSsmDesc, dict(n_seqs=2, n_slots=4, h_qk=2, h_v=4, d_k=128, d_v=64, dtype=1, softplus=1,
                                           total_tokens=2, total_out_tokens=2, x_stride=256, b_stride=256,
                                           c_stride=256, dt_stride=4, y_stride=256), kw)


def _paged(gdn, **kw):
    return _fill(gdn._lib.GdnPagedDesc, dict(n_seqs=2, h_q=8, h_kv=2, d=128, dtype=1, page_size=16, n_pages=10,
                                             max_pages=5, max_kv_len=80, rot_dim=64, interleaved=0, norm=1,
                                             max_pos=80, eps=1e-6, scale=0.1, total_tokens=6, q_stride=1024,
                                             k_stride=256, v_stride=256, o_stride=1024, page_stride=16 * 256,
                                             token_stride=256, head_stride=128), kw)


def _call(gdn, name, desc, n, change=None, ws=P, ws_bytes=BIG):
    args = [P] * n
    for i, v in (change or {}).items():
        args[i] = v
    return getattr(gdn.load(), name)(ctypes.byref(desc) if desc is not None else None, *args, ws, ws_bytes, None)


N = {"gdn_conv": 7, "gdn_conv_step": 6, "gdn_ssm_scan": 13, "gdn_ssm_step": 10, "gdn_qk_norm_rope": 13,
     "gdn_paged_attn": 8}
MAKE = {"gdn_conv": _conv, "gdn_conv_step": _conv, "gdn_ssm_scan": _ssm, "gdn_ssm_step": _ssm,
        "gdn_qk_norm_rope": _paged, "gdn_paged_attn": _paged}
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 6

DESC_ERRORS = [
    ("gdn_conv", dict(dtype=2), DTYPE), ("gdn_conv", dict(n_seqs=-1), SHAPE), ("gdn_conv", dict(silu=2), SHAPE),
    ("gdn_conv", dict(channels=0), SHAPE), ("gdn_conv", dict(width=1), UNSUPPORTED),
    ("gdn_conv", dict(width=5), UNSUPPORTED), ("gdn_conv", dict(channels=60, x_stride=60, y_stride=60), ALIGN),
    ("gdn_conv", dict(x_stride=56), ALIGN), ("gdn_conv", dict(y_stride=68), ALIGN),
    ("gdn_conv", dict(total_tokens=1 << 31), SHAPE),
    ("gdn_conv_step", dict(total_tokens=3), SHAPE), ("gdn_conv_step", dict(n_slots=-1), SHAPE),
    ("gdn_ssm_scan", dict(h_v=3), SHAPE), ("gdn_ssm_scan", dict(d_k=96), UNSUPPORTED),
    ("gdn_ssm_scan", dict(d_v=32), UNSUPPORTED), ("gdn_ssm_scan", dict(dtype=-1), DTYPE),
    ("gdn_ssm_scan", dict(total_out_tokens=3), SHAPE), ("gdn_ssm_scan", dict(x_stride=255), ALIGN),
    ("gdn_ssm_scan", dict(c_stride=0), ALIGN), ("gdn_ssm_scan", dict(dt_stride=3), SHAPE),
    ("gdn_ssm_scan", dict(softplus=5), SHAPE),
    ("gdn_ssm_step", dict(total_tokens=5), SHAPE), ("gdn_ssm_step", dict(y_stride=252), ALIGN),
    ("gdn_qk_norm_rope", dict(rot_dim=24), SHAPE), ("gdn_qk_norm_rope", dict(rot_dim=144), SHAPE),
    ("gdn_qk_norm_rope", dict(interleaved=2), SHAPE), ("gdn_qk_norm_rope", dict(eps=-1.0), SHAPE),
    ("gdn_qk_norm_rope", dict(eps=float("nan")), SHAPE), ("gdn_qk_norm_rope", dict(k_stride=128), ALIGN),
    ("gdn_qk_norm_rope", dict(head_stride=64), ALIGN),
    ("gdn_paged_attn", dict(h_q=7), SHAPE), ("gdn_paged_attn", dict(d=96), UNSUPPORTED),
    ("gdn_paged_attn", dict(page_size=0), SHAPE), ("gdn_paged_attn", dict(max_kv_len=-1), SHAPE),
    ("gdn_paged_attn", dict(max_kv_len=(1 << 30) + 1), SHAPE), ("gdn_paged_attn", dict(scale=float("inf")), SHAPE),
    ("gdn_paged_attn", dict(token_stride=120), ALIGN), ("gdn_paged_attn", dict(page_stride=4), ALIGN),
    ("gdn_paged_attn", dict(total_tokens=1 << 29), SHAPE), ("gdn_paged_attn", dict(o_stride=1020), ALIGN),
]


@pytest.mark.parametrize("name,change,code", DESC_ERRORS)
def test_descriptor_refusals(gdn, name, change, code):
    assert _call(gdn, name, MAKE[name](gdn, **change), N[name]) == code


OPTIONAL = {"gdn_conv": {2, 4, 5}, "gdn_conv_step": {2, 4}, "gdn_ssm_scan": {5, 6, 8, 9, 11, 12},
            "gdn_ssm_step": {5, 6, 8}, "gdn_qk_norm_rope": {3, 4, 9}, "gdn_paged_attn": {7}}
# pointers that only need the alignment of their elements
NARROW = {"gdn_conv": {1, 2, 3}, "gdn_conv_step": {1, 2, 4}, "gdn_ssm_scan": {3, 4, 5, 6, 7, 8, 12},
          "gdn_ssm_step": {3, 4, 5, 6, 8}, "gdn_qk_norm_rope": {3, 4, 5, 6, 7, 8, 9}, "gdn_paged_attn": {3, 4, 5, 7}}


@pytest.mark.parametrize("name", sorted(N))
def test_pointer_refusals(gdn, name):
    d = MAKE[name](gdn)
    odd = ctypes.c_void_p(0x100001)
    for i in range(N[name]):
        if i not in OPTIONAL[name]:
            assert _call(gdn, name, d, N[name], {i: None}) == NULL, i
        assert _call(gdn, name, d, N[name], {i: odd if i in NARROW[name] else PM}) == ALIGN, i
    assert _call(gdn, name, None, N[name]) == NULL
    assert _call(gdn, name, d, N[name], ws=None) == NULL
    assert _call(gdn, name, d, N[name], ws=PM) == ALIGN
    assert _call(gdn, name, d, N[name], ws_bytes=255) == WORKSPACE


@pytest.mark.parametrize("name", sorted(N))
def test_nothing_to_do_is_accepted(gdn, name):
    zero = dict(n_seqs=0, total_tokens=0)
    if MAKE[name] is _ssm:
        zero["total_out_tokens"] = 0
    assert _call(gdn, name, MAKE[name](gdn, **zero), N[name], ws_bytes=256) == 0


def test_fewer_slots_than_rows(gdn):
    assert _call(gdn, "gdn_conv_step", _conv(gdn, n_slots=1), 6, {4: None}) == SHAPE
    assert _call(gdn, "gdn_ssm_step", _ssm(gdn, n_slots=1), 10, {8: None}) == SHAPE


def test_workspace_sizes(gdn):
    # few long sequences are cut: the states of the segments
    d = _ssm(gdn, n_seqs=1, h_v=32, h_qk=2, total_tokens=32768, total_out_tokens=32768, x_stride=2048, y_stride=2048, dt_stride=32)
    need = gdn.gdn_ssm_workspace_bytes(d)
    assert need > 256 and _call(gdn, "gdn_ssm_scan", d, 13, ws_bytes=need - 1) == WORKSPACE
    assert gdn.gdn_ssm_workspace_bytes(_ssm(gdn)) == 256
    assert gdn.gdn_ssm_workspace_bytes(_ssm(gdn, d_k=96)) == 0
    d = _paged(gdn, max_kv_len=65536, max_pages=4096)
    need = gdn.gdn_paged_workspace_bytes(d)
    assert need > 256 and _call(gdn, "gdn_paged_attn", d, 8, ws_bytes=need - 1) == WORKSPACE
    assert gdn.gdn_paged_workspace_bytes(_paged(gdn, max_kv_len=1)) == 256
    assert gdn.gdn_paged_workspace_bytes(_paged(gdn, d=80)) == 0


@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_sizes_of_any_shape(gdn, dtype):
    # the plans behind them, from nothing to the largest sizes: at most a row's part for every 64 keys,
    # a state for every chunk of 64 tokens
    r = random.Random(dtype)
    for _ in range(3000):
        n, total = r.choice([0, 1, 2, 17, 300, 100000]), r.choice([0, 1, 5, 64, 1000, 70000, 1 << 24])
        h_kv, G, d = r.choice([1, 2, 8]), r.choice([1, 3, 8, 32]), r.choice([64, 128, 256])
        kv = r.choice([0, 1, 63, 64, 257, 4095, 4096, 100001, 1 << 30])
        if total * h_kv * G <= 0x7fffffff:
            s = _paged(gdn, n_seqs=n, total_tokens=total, h_q=h_kv * G, h_kv=h_kv, d=d, max_kv_len=kv, dtype=dtype,
                       token_stride=2048, head_stride=256, page_stride=32768)
            need, part = gdn.gdn_paged_workspace_bytes(s), total * h_kv * G * (d + 2) * 4
            assert 256 <= need <= 512 + part * max(1, -(-kv // 64)), (n, total, h_kv, G, d, kv)
        k, v = r.choice([64, 128]), r.choice([64, 128])
        s = _ssm(gdn, n_seqs=n, h_qk=h_kv, h_v=h_kv * G, d_k=k, d_v=v, total_tokens=total, total_out_tokens=total, dtype=dtype,
                 x_stride=h_kv * G * v, y_stride=h_kv * G * v, b_stride=h_kv * k, c_stride=h_kv * k, dt_stride=h_kv * G)
        state = n * h_kv * G * (k * v + 1) * 4
        assert 256 <= gdn.gdn_ssm_workspace_bytes(s) <= 512 + state * max(1, -(-total // 64)), (n, total, h_kv, G, k, v)


def test_gated_delta_step_refusals(gdn):
    L = gdn._lib

    def call(n_slots=2, slots=P, q=P, ws=P, **kw):
        d = _fill(L.GdnDesc, dict(n_seqs=2, h_qk=2, h_v=4, d_k=128, d_v=128, qkv_dtype=1, o_dtype=1, scale=1.0,
                                  total_tokens=2, total_out_tokens=2), kw)
        return gdn.load().gdn_step(ctypes.byref(d), q, P, P, P, P, P, n_slots, slots, P, ws, 256, None)

    assert call(h_v=3) == SHAPE and call(total_tokens=3) == SHAPE and call(n_slots=-1) == SHAPE
    assert call(n_slots=1, slots=None) == SHAPE
    assert call(d_k=32) == UNSUPPORTED and call(qkv_dtype=9) == DTYPE and call(qkv_dtype=0, o_dtype=1) == DTYPE
    assert call(q=None) == NULL and call(q=PM) == ALIGN and call(ws=None) == NULL
    assert call(n_seqs=0, total_tokens=0, total_out_tokens=0) == 0


# ------------------------------------------------------------------ the Python binding
def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


def _refused(gdn, code, f, *a, **kw):
    with pytest.raises(gdn.GdnError) as e:
        f(*a, **kw)
    assert e.value.code == code, str(e.value)


def test_python_conv_refusals(gdn):
    x, w, cu = _z(6, 64), _z(64, 4, dtype=torch.float32), _i(0, 2, 6)
    _refused(gdn, DTYPE, gdn.gdn_conv, x.half(), w, cu)
    _refused(gdn, DTYPE, gdn.gdn_conv, x, w.bfloat16(), cu)
    _refused(gdn, DTYPE, gdn.gdn_conv, x, w, cu.long())
    _refused(gdn, SHAPE, gdn.gdn_conv, x, w[:32], cu)
    _refused(gdn, SHAPE, gdn.gdn_conv, x, w, cu, state0=_z(2, 2, 64))
    _refused(gdn, DTYPE, gdn.gdn_conv, x, w, cu, state0=_z(2, 3, 64, dtype=torch.float32))
    _refused(gdn, ALIGN, gdn.gdn_conv, _z(64, 6).t(), w, cu)
    _refused(gdn, SHAPE, gdn.gdn_conv, x, w, cu, activation="relu")
    _refused(gdn, SHAPE, gdn.gdn_conv, x, w, cu)                        # on the CPU
    _refused(gdn, SHAPE, gdn.gdn_conv_step, x, w, _z(9, 2, 64))
    _refused(gdn, SHAPE, gdn.gdn_conv_step, x, w, _z(9, 3, 64), slots=_i(0, 1))


def test_python_ssm_refusals(gdn):
    f = torch.float32
    x, B, dt, A, cu = _z(6, 4, 64), _z(6, 2, 128), _z(6, 4), _z(4, dtype=f), _i(0, 2, 6)
    _refused(gdn, SHAPE, gdn.gdn_ssm_scan, x, B, B[:5], dt, A, cu)
    _refused(gdn, DTYPE, gdn.gdn_ssm_scan, x, B, B, dt.float(), A, cu)
    _refused(gdn, SHAPE, gdn.gdn_ssm_scan, x, B, B, dt, _z(5, dtype=f), cu)
    _refused(gdn, SHAPE, gdn.gdn_ssm_scan, x, B, B, dt, A, cu, r=_i(1, 1))          # no total_out_tokens
    _refused(gdn, SHAPE, gdn.gdn_ssm_scan, x, B, B, dt, A, cu, S0=_z(2, 4, 64, 128, dtype=f))
    _refused(gdn, SHAPE, gdn.gdn_ssm_scan, x, B, B, dt, A, cu)
    _refused(gdn, SHAPE, gdn.gdn_ssm_step, x, B, B, dt, A, _z(9, 4, 128, 128, dtype=f))
    _refused(gdn, DTYPE, gdn.gdn_ssm_step, x, B, B, dt, A, _z(9, 4, 128, 64))
    q, v, g = _z(6, 2, 128), _z(6, 4, 64), _z(6, 4, dtype=f)
    _refused(gdn, DTYPE, gdn.gdn_step, q, q, v, g.bfloat16(), g, _z(9, 4, 128, 64, dtype=f))
    _refused(gdn, SHAPE, gdn.gdn_step, q, q, v, g, g, _z(9, 4, 64, 64, dtype=f))


def test_python_paged_refusals(gdn):
    f = torch.float32
    q, k, kc, table, cu, kv = _z(6, 8, 128), _z(6, 2, 128), _z(10, 16, 2, 128), _i(1, 2, 3, 4).view(2, 2), _i(0, 2, 6), _i(20, 30)
    cs = _z(32, 64, dtype=f)
    _refused(gdn, SHAPE, gdn.gdn_paged_attn, q, kc, kc[:9], table, cu, kv)
    _refused(gdn, DTYPE, gdn.gdn_paged_attn, q, kc.float(), kc.float(), table, cu, kv)
    _refused(gdn, SHAPE, gdn.gdn_paged_attn, _z(6, 8, 64), kc, kc, table, cu, kv)
    _refused(gdn, SHAPE, gdn.gdn_paged_attn, q, kc, kc, table[:1], cu, kv)
    _refused(gdn, DTYPE, gdn.gdn_paged_attn, q, kc, kc, table, cu, kv.long())
    _refused(gdn, SHAPE, gdn.gdn_paged_attn, q, kc, kc, table, cu, kv, lse=_z(8, 6, dtype=f))
    _refused(gdn, SHAPE, gdn.gdn_paged_attn, q, kc, kc, table, cu, kv)
    _refused(gdn, SHAPE, gdn.gdn_qk_norm_rope, q, k[:5], k, cs, kc, kc, table, cu, kv)
    _refused(gdn, DTYPE, gdn.gdn_qk_norm_rope, q, k, k, cs.bfloat16(), kc, kc, table, cu, kv)
    _refused(gdn, SHAPE, gdn.gdn_qk_norm_rope, q, k, k, cs, kc, kc, table, cu, kv, q_weight=_z(64, dtype=f))
    _refused(gdn, SHAPE, gdn.gdn_qk_norm_rope, q, k, k, cs, kc, kc, table, cu, kv, positions=_i(1, 2))


# ------------------------------------------------------------------ index arithmetic
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "gdn_index.h"
using namespace gdn;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main()
{
    srand(7);
    // every row of every sequence is in exactly one tile of that sequence, and the tiles fit
    for (int round = 0; round < 400; ++round) {
        const int n = 1 + rand() % 9, mul = 1 + rand() % 12, tile = 1 << (rand() % 9);
        std::vector<int32_t> cu(n + 1, 0);
        for (int i = 0; i < n; ++i) cu[i + 1] = cu[i] + (rand() % 3 ? rand() % 300 : 0);
        const int64_t all = (int64_t)cu[n] * mul / tile + n;
        for (int i = 0; i < n; ++i) {
            const int64_t f = first_tile(cu[i], i, mul, tile), next = i + 1 < n ? first_tile(cu[i + 1], i + 1, mul, tile) : all;
            const int64_t rows = (int64_t)(cu[i + 1] - cu[i]) * mul;
            CHECK(next - f >= 1 && (next - f) * tile >= rows);
        }
    }
    CHECK(first_tile(2000000000, 3, 64, 16) == 8000000003LL);
    CHECK(range_ok(0, 0, 0) && range_ok(3, 9, 9) && !range_ok(-1, 4, 9) && !range_ok(5, 4, 9) && !range_ok(0, 10, 9));
    CHECK(kv_ok(0, 80, 16, 0) && kv_ok(80, 80, 16, 5) && !kv_ok(80, 80, 16, 4) && !kv_ok(81, 80, 16, 9) && !kv_ok(-1, 80, 16, 9));
    CHECK(!kv_ok(2147483647, 1 << 30, 16, 2147483647) && kv_ok(1 << 30, 1 << 30, 1, 1 << 30));
    const int32_t table[4] = {7, -1, 10, 9};
    bool bad = false;
    CHECK(cache_offset(table, 5, 16, 10, 4096, 256, bad) == 7 * 4096 + 5 * 256 && !bad);
    CHECK(cache_offset(table, 63, 16, 10, 1LL << 33, 256, bad) == 9 * (1LL << 33) + 15 * 256 && !bad);
    CHECK(cache_offset(table, 16, 16, 10, 4096, 256, bad) == -1 && bad);
    bad = false;
    CHECK(cache_offset(table, 47, 16, 10, 4096, 256, bad) == -1 && bad);
    puts("index arithmetic: ok");
    return 0;
}
"""


@pytest.mark.parametrize("san", [None, "address,undefined"])
def test_index_arithmetic(tmp_path, san):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "index.cpp", str(tmp_path / "index")
    src.write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "gated_deltanet_state_gdn_amd", "csrc"), str(src), "-o", exe]
    subprocess.check_call(cmd + (["-fsanitize=" + san] if san else []))
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and "ok" in p.stdout, p.stdout + p.stderr
