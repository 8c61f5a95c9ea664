"""GPU: the suffix and decode operators at the ends of their types, and the roundings that they state."""
import ctypes
import math

import pytest
import torch

import ops_reference as R
from gpu_helpers import say
from test_gpu_ops import BF, F32, TYPES, Cache, G, Rand, attn_check, ints, new_ws, scan_check, scan_inputs

pytestmark = pytest.mark.gpu


@TYPES
def test_gates_of_the_types_ends(dt):
    """softplus at the type's lowest value is 0: the token leaves the state as it is (a masked token).  At its
    highest, with B = x = 0, the token clears the state.  Both are finite and stay out of their neighbours."""
    g, h, k, p, T = 1, 2, 64, 64, 200
    r = Rand(13)
    inp = {n: t.contiguous() for n, t in scan_inputs(r, T, g, h, k, p, dt, True).items()}
    low, high = torch.finfo(dt).min, torch.finfo(dt).max
    inp["dt"][[0, 3, 64, 70, 199]] = low
    inp["dt"][[10, 11], 0] = -200.0
    inp["dt"][12, 1] = -1e30
    for t in (40, 130):
        inp["dt"][t] = high
        inp["B"][t], inp["x"][t] = 0, 0
    S0 = r.n(1, h, k, p)
    S, y, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints([0, T]), S0=S0)
    scan_check(y, S[0], 0, inp, 0, T, R.d(S0[0]), dt, True, "gates")
    # the same values in the single-token form, a row each
    rows = [0, 10, 12, 40, 41]
    pool = r.n(len(rows), h, k, p)
    before = pool.clone()
    a = [inp[n][rows].contiguous() for n in ("x", "B", "C", "dt")]
    y = G().gdn_ssm_step(*a, inp["A"], pool, D=inp["D"], dt_bias=inp["dt_bias"])
    for i in range(len(rows)):
        ref = R.ssm_tokens(*(R.d(t[i:i + 1]) for t in a), R.d(inp["A"]), R.d(inp["D"]), R.d(inp["dt_bias"]), R.d(before[i]))
        R.within(pool[i], ref[2], 20 * R.U32 * ref[3] + 1e-30, "S of row %d" % i)
        R.within(y[i:i + 1], ref[0], R.u(dt) * ref[0].abs() + (30 + k) * R.U32 * ref[1] + 1e-30, "y of row %d" % i)
    # NaN stays NaN
    inp["dt"][5, 0] = math.nan
    S, y, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints([0, T]), S0=S0)
    assert y[5, 0].isnan().all() and S[0, 0].isnan().all() and not S[0, 1].isnan().any() and not y[:, 1].isnan().any()
    nan = inp["dt"][5:6].contiguous()
    pool = before[:1].clone()
    y = G().gdn_ssm_step(*(inp[n][5:6].contiguous() for n in ("x", "B", "C")), nan, inp["A"], pool, D=inp["D"], dt_bias=inp["dt_bias"])
    assert y[0, 0].isnan().all() and pool[0, 0].isnan().all() and not y[0, 1].isnan().any()


@pytest.mark.parametrize("step", [False, True])
def test_silu_in_fp32(step):
    """SiLU of known arguments (the taps are zero, the bias is the argument).  Roundings: the exponential (2, and
    3 of its argument's), 1 + z, the reciprocal (2), two products, each at most one: 10 halves of a step; the
    exponential is 0 below 2^-126, which is worth |y| 2^-126."""
    arg = torch.cat([torch.linspace(-100, 100, 4001), torch.tensor([0.0, -1e-30, 1e-30, 3e38, -3e38, -87.3, -87.4])]).cuda()
    arg = torch.cat([arg, torch.zeros(-arg.numel() % 4, device="cuda")])
    ch = arg.numel()
    x, w = Rand(2).n(3, ch), torch.zeros(ch, 2, device="cuda")
    if step:
        y = G().gdn_conv_step(x, w, torch.zeros(3, 1, ch, device="cuda"), bias=arg)
    else:
        y, _ = G().gdn_conv(x, w, ints([0, 3]), bias=arg)
    a = R.d(arg)
    ref = torch.where(a < -700, torch.zeros_like(a), a * torch.sigmoid(a.clamp(min=-700)))
    R.within(y, ref.expand(3, -1), 10 * R.U32 * ref.abs() + 90 * 2.0 ** -126, "SiLU")


@pytest.mark.parametrize("k,p,h", [(64, 64, 32), (64, 128, 32), (128, 64, 15), (128, 64, 32), (128, 128, 16)])
def test_scan_in_segments_rounds_the_state_once(k, p, h):
    """bf16, cut into segments: M and S are rounded to bf16 for their products with x and C, and nothing else
    is.  Gates of 1 + 2^-7, no decay, and inputs 1 + j 2^-7 (40 <= j < 64): the state's terms dt x lie j 2^-14
    above a bf16 value, so that rounding them to bf16 would make every state, and y, smaller by
    j 2^-14 / (1 + j 2^-7), 1.5e-3 and more.  The roundings of S and M have no common sign: of at least 2^13 of them, 2^-8
    at most, the mean is beyond 2^-11 with a probability below 1e-12 (Hoeffding: 2 exp(-2^13 / (2 * 64)))."""
    r = Rand(k + p)
    T = 8192
    x = (1 + torch.randint(40, 64, (T, h, p), generator=r.g) * 2.0 ** -7).cuda().to(BF)
    B, C = r.n(T, 1, k, dt=BF), r.n(T, 1, k, dt=BF)
    dt = torch.full((T, h), 1 + 2.0 ** -7, dtype=BF, device="cuda")
    A = torch.zeros(h, device="cuda")
    need = G().gdn_ssm_workspace_bytes(G().make_ssm_desc(x, B, 1))
    segs = (need - 256) // (h * (k * p + 1) * 4)
    assert segs > 1
    per = -(-(T // 64) // segs) * 64
    say("scan in", segs, "segments of", per)
    assert per >= 128
    S, y, _ = G().gdn_ssm_scan(x, B, C, dt, A, ints([0, T]), softplus=False, ws=new_ws(need))
    xs = x.double() * dt.double()[..., None]
    ref = torch.empty(T, h, p, dtype=torch.float64, device="cuda")
    low = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    M = torch.where(low, C[:, 0].double() @ B[:, 0].double().t(), torch.zeros((), dtype=torch.float64, device="cuda"))
    for i in range(h):
        ref[:, i] = M @ xs[:, i]
    # rows whose state comes from their own segment in part: all but a segment's first chunk; in the first one all of it does
    got, want = y[64:per].double(), ref[64:per]
    bias = float((got * want).sum() / (want * want).sum()) - 1
    say("  common part of the outputs' error %.2e" % bias)
    assert abs(bias) <= 2.0 ** -11


@TYPES
@pytest.mark.parametrize("n,hk,bound", [(1100, 8, 1 << 30), (600, 8, 1 << 30), (2, 2, 1 << 30), (1100, 8, 1 << 27)])
def test_attention_under_the_loosest_bound(dt, n, hk, bound):
    """max_kv_len as large as it may be, beside few cached tokens: the C call, whose bound no table limits."""
    g, r, hq, dim, ps = G(), Rand(n), 2 * hk, 64, 16
    kv = [1 + (7 * i) % 20 for i in range(n)]
    kv[-1] = 45
    c = Cache(r, kv, ps, hk, dim, dt)
    q, o, lse = r.n(n, hq, dim, dt=dt), torch.full((n, hq, dim), 7.0, dtype=dt, device="cuda"), torch.empty(n, hq, device="cuda")
    d = g.make_paged_desc(q, c.k, c.table, n)
    d.max_kv_len = bound
    need = g.gdn_paged_workspace_bytes(d)
    say("attention under a bound of", bound, dt, n, hk, "workspace", need)
    assert 256 <= need <= 1 << 30
    ws, cu, kvt = new_ws(need), ints(list(range(n + 1))), ints(kv)
    p = [ctypes.c_void_p(t.data_ptr()) for t in (q, c.k, c.v, c.table, cu, kvt, o, lse, ws)]
    code = g.load().gdn_paged_attn(ctypes.byref(d), *p, need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert code == 0 and g.gdn_device_status(ws) == 0
    some = [0, 1, n // 2, n - 1]
    part = Cache.__new__(Cache)
    part.keys, part.vals = [c.keys[i] for i in some], [c.vals[i] for i in some]
    attn_check(part, q[some], o[some], lse[some], [1] * len(some), [kv[i] for i in some], dim ** -0.5, dt)
    assert not o.isnan().any() and not lse.isnan().any()
