"""GPU: forms of the kernels that only larger or other sizes than those of test_gpu_ops.py reach, by the same
checks against the 64-bit reference and with the same tolerances."""
import pytest

import test_gpu_ops as ops
from test_gpu_ops import BF, F32, TYPES, _gpu  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@TYPES
@pytest.mark.parametrize("ch,W,lens,start,silu,bias", [
    (4104, 4, [900], True, True, True), (4104, 3, [850, 1, 0, 40], False, True, False),
    (64, 2, [3] * 519 + [400], True, False, True), (72, 4, [0, 2, 90] * 171, True, True, True),
])
def test_conv_of_many_workgroups(dt, ch, W, lens, start, silu, bias):
    # 512 workgroups and more: sixteen tokens a thread
    ops.test_conv(dt, ch, W, lens, start, silu, bias)


@TYPES
@pytest.mark.parametrize("g,h,k,p,lens,start", [
    (1, 3, 128, 64, [700], True), (1, 2, 128, 128, [300], False),        # workgroups of 64 columns
    (2, 16, 128, 64, [700, 0, 290, 610], True), (2, 16, 128, 128, [1100, 400], True),    # bf16: of 128
])
def test_scan_in_segments(dt, g, h, k, p, lens, start):
    ops.test_scan(dt, g, h, k, p, lens, start, True)


@pytest.mark.parametrize("dt,hq,hk,dim,ps,lens,ctx", [
    # few rows over long contexts: two waves a workgroup; 16 rows, and 32
    (BF, 16, 2, 256, 64, [1, 1, 1, 1], [4999, 70, 1200, 300]),
    (BF, 48, 2, 256, 64, [1] * 30, [0, 4099, 3] + [64 + i for i in range(25)] + [2100, 900]),
    # many rows, 128 to a workgroup; fp32 of 128
    (BF, 4, 2, 256, 16, [40], [260]), (BF, 4, 2, 256, 24, [37, 0, 60], [803, 5, 1]), (F32, 8, 2, 128, 16, [100, 200], [600, 9]),
    # joined in one slice: up to eight splits of many rows
    (F32, 16, 4, 64, 16, [200, 1, 0, 99, 100, 150, 50, 64, 30, 6], [305, 9, 4, 0, 105, 1, 64, 3, 0, 41]),
    (F32, 16, 4, 128, 16, [200, 1, 0, 99, 100, 150, 50, 64, 30, 6], [305, 9, 4, 0, 105, 1, 64, 3, 0, 41]),
    (BF, 8, 2, 128, 16, [300, 260], [400, 100]), (BF, 8, 2, 128, 16, [520], [380]),
])
def test_attention_forms(dt, hq, hk, dim, ps, lens, ctx):
    ops.test_attention(dt, hq, hk, dim, ps, lens, ctx, False)
