"""GPU: the suffix and decode operators against plain 64-bit implementations (ops_reference.py).

Tolerances count roundings.  One rounding is off by at most u = eps / 2 of its type relative to the
value; a result that passes n roundings of type t along its longest path is off by at most n u times
the sum of the absolute values behind it (abs, from the reference).  The counts are stated where
they are used, before the first run of the kernels.
"""
import math

import pytest
import torch

import ops_reference as R
from gpu_helpers import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import gated_deltanet_state_gdn_amd as gdn
    gdn.load()
    yield


def G():
    import gated_deltanet_state_gdn_amd as gdn
    return gdn


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def n(self, *shape, dt=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(dt).cuda()

    def perm(self, n):
        return torch.randperm(n, generator=self.g)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def new_ws(n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ convolution
CONV = [  # channels, width, lengths, state0, silu, bias
    (128, 4, [1], True, True, True), (136, 2, [0, 5, 1, 0, 2, 70], True, True, False),
    (8, 3, [33, 0, 1, 4100], False, False, True), (2056, 4, [17, 64, 3], True, True, True),
    (512, 4, [600, 1, 2, 3, 4, 0], False, True, True), (72, 4, [0, 0], True, True, True),
]


def conv_tol(y, ab, dt, W):
    # W products and sums, the bias, then SiLU (exponential, sum, quotient: 8 roundings; its slope
    # is at most 1.1), and the rounding to the type
    return R.u(dt) * y.abs() + (2 * W + 10) * 1.1 * R.U32 * ab + 1e-30


@TYPES
@pytest.mark.parametrize("ch,W,lens,start,silu,bias", CONV)
def test_conv(dt, ch, W, lens, start, silu, bias):
    r = Rand(ch + W)
    cu = cu_of(lens)
    T, n, behind = cu[-1], len(lens), 3                       # rows behind the last sequence
    wide = r.n(T + behind, ch + 16, dt=dt)
    x, w = wide[:, 8:8 + ch], r.n(ch, W)
    b = r.n(ch) if bias else None
    s0 = r.n(n, W - 1, ch, dt=dt) if start else None
    y = torch.full((T + behind, ch), 7.0, dtype=dt, device="cuda")
    ws = new_ws()
    say("conv", dt, ch, W, lens)
    _, so = G().gdn_conv(x, w, ints(cu), bias=b, state0=s0, activation="silu" if silu else None, y=y, ws=ws)
    assert G().gdn_device_status(ws) == 0
    assert (y[T:] == 7).all()
    for i in range(n):
        old = R.d(s0[i]) if start else torch.zeros(W - 1, ch, dtype=torch.float64)
        ref, ab, last = R.conv_tokens(R.d(x[cu[i]:cu[i + 1]]), R.d(w), R.d(b) if bias else None, old, silu)
        R.within(y[cu[i]:cu[i + 1]], ref, conv_tol(ref, ab, dt, W), "y of sequence %d" % i)
        assert torch.equal(R.d(so[i]), last)
    if start:                                                  # the new state in place of the old one
        G().gdn_conv(x, w, ints(cu), bias=b, state0=s0, state_out=s0, activation="silu" if silu else None, y=y, ws=ws)
        assert torch.equal(s0, so)


@TYPES
@pytest.mark.parametrize("ch,W,rows", [(8, 2, 1), (520, 4, 7), (2048, 3, 130)])
def test_conv_step(dt, ch, W, rows):
    r = Rand(rows)
    x, w, b = r.n(rows, ch + 8, dt=dt)[:, 8:], r.n(ch, W), r.n(ch)
    pool = r.n(rows + 3, W - 1, ch, dt=dt)
    slots = r.perm(rows + 3)[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1                                          # a padded row
    before, y, ws = pool.clone(), torch.full((rows, ch), 7.0, dtype=dt, device="cuda"), new_ws()
    say("conv_step", dt, ch, W, rows)
    G().gdn_conv_step(x, w, pool, slots=slots.cuda(), bias=b, y=y, ws=ws)
    assert G().gdn_device_status(ws) == 0
    want = R.d(before)
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            assert (y[i] == 7).all()
            continue
        ref, ab, want[s] = R.conv_tokens(R.d(x[i:i + 1]), R.d(w), R.d(b), R.d(before[s]), True)
        R.within(y[i:i + 1], ref, conv_tol(ref, ab, dt, W), "y of row %d" % i)
    assert torch.equal(R.d(pool), want)


# ------------------------------------------------------------------ state space scan
SCAN = [  # groups, heads, d_k, d_v, lengths, state0, softplus
    (1, 1, 64, 64, [1], True, True), (1, 2, 128, 64, [65, 0, 64, 1, 130], True, True),
    (2, 4, 64, 128, [63, 200], False, True), (2, 2, 128, 128, [129], True, False),
    (1, 4, 64, 64, [1100], True, True),                        # cut into segments
    # workgroups of 128 columns (bf16): in one launch, and cut into segments with empty ones among them
    (2, 8, 64, 64, [3, 65, 0, 17, 64, 1, 30, 128] * 8, True, True), (1, 16, 128, 128, [1, 66, 0, 5] * 4 + [9], False, True),
    (2, 32, 64, 64, [2600, 0, 5, 1500], True, True), (4, 16, 64, 128, [2500, 1700], True, True),
    (3, 9, 64, 64, [20] * 60, False, True),                    # many workgroups, but three heads to a group
    (2, 2, 128, 128, [0, 0], True, True),                      # nothing to scan: the states pass through
]


def scan_inputs(r, T, g, h, k, p, dt, softplus):
    wide = r.n(T, h * p + 2 * g * k + 16, dt=dt)
    x = wide[:, :h * p].unflatten(1, (h, p))
    B = wide[:, h * p:h * p + g * k].unflatten(1, (g, k))
    C = wide[:, h * p + g * k:h * p + 2 * g * k].unflatten(1, (g, k))
    dtr = r.n(T, h + 1, dt=dt)
    if not softplus:
        dtr = dtr.abs() * 0.1
    A = -torch.rand(h, generator=r.g).cuda() * 8 - 0.05
    return dict(x=x, B=B, C=C, dt=dtr[:, 1:], A=A, D=r.n(h), dt_bias=r.n(h, scale=0.5) - 2 if softplus else r.n(h).abs() * 0.1)


def scan_tols(y, ya, S, Sa, dt, L):
    # state: a 64-term sum per chunk (bf16: three terms each), and per chunk behind it the decay's
    # exponential (4 roundings at an exponent of O(1)), product and sum; the token's gate (softplus,
    # exponent: 8 roundings)
    chunks = L // 64 + 1
    st = (3 * 64 + 40 + 8 * chunks) * R.U32 * Sa + 1e-30
    # y: the roundings of M and of S (bf16), the fp32 sums over 128 and 64 terms with the state's own,
    # and the final one
    mid = 2 * R.u(dt) if dt is BF else 0.0
    yt = R.u(dt) * y.abs() + (mid * (1 + 1 / 64) + (128 + 64 * 3 + 40 + 8 * chunks) * R.U32) * ya + 1e-30
    return yt, st


def scan_check(got_y, got_S, i, inp, lo, hi, S0, dt, softplus, what):
    ref = R.ssm_tokens(*(R.d(inp[k][lo:hi]) for k in ("x", "B", "C", "dt")), R.d(inp["A"]), R.d(inp["D"]),
                       R.d(inp["dt_bias"]), S0, softplus)
    yt, st = scan_tols(*ref, dt, hi - lo)
    if got_y is not None:
        R.within(got_y, ref[0], yt, what + ": y")
    R.within(got_S, ref[2], st, what + ": S")
    return ref, st


@TYPES
@pytest.mark.parametrize("g,h,k,p,lens,start,softplus", SCAN)
def test_scan(dt, g, h, k, p, lens, start, softplus):
    r = Rand(k + p + len(lens))
    cu, n = cu_of(lens), len(lens)
    T = cu[-1]
    inp = scan_inputs(r, T + 2, g, h, k, p, dt, softplus)
    S0 = r.n(n, h, k, p) if start else None
    y = torch.full((T + 2, h, p), 7.0, dtype=dt, device="cuda")
    desc = G().make_ssm_desc(inp["x"], inp["B"], n)
    ws = new_ws(G().gdn_ssm_workspace_bytes(desc))
    say("scan", dt, g, h, k, p, lens, "workspace", ws.numel())
    S, _, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints(cu), softplus=softplus, S0=S0, y_out=y, ws=ws)
    assert G().gdn_device_status(ws) == 0
    assert (y[T:] == 7).all()
    zero = torch.zeros(h, k, p, dtype=torch.float64)
    refs = [scan_check(y[cu[i]:cu[i + 1]], S[i], i, inp, cu[i], cu[i + 1], R.d(S0[i]) if start else zero, dt, softplus,
                       "sequence %d" % i) for i in range(n)]
    S2, none, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints(cu), softplus=softplus, S0=S0, y_out=None, ws=ws)
    assert none is None
    for i, (ref, st) in enumerate(refs):
        R.within(S2[i], ref[2], st, "state alone %d" % i)
    if start:                                                  # the new state in place of the old one
        G().gdn_ssm_scan(**inp, cu_seqlens=ints(cu), softplus=softplus, S0=S0, S_out=S0, y_out=y, ws=ws)
        assert torch.equal(S0, S)


@TYPES
@pytest.mark.parametrize("lens,rep", [([200, 70, 5, 90], [130, 0, 5, 64]), ([1500], [1201])])
def test_scan_windows(dt, lens, rep):
    g, h, k, p = 1, 2, 64, 64
    r = Rand(5)
    cu, n = cu_of(lens), len(lens)
    inp = scan_inputs(r, cu[-1], g, h, k, p, dt, True)
    cu_out, ws = torch.full((n + 1,), -7, dtype=torch.int32, device="cuda"), new_ws(1 << 22)
    say("scan windows", dt, lens, rep)
    S, y, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints(cu), r=ints(rep), total_out_tokens=sum(rep), cu_out=cu_out, ws=ws)
    assert G().gdn_device_status(ws) == 0 and cu_out.tolist() == cu_of(rep)
    at = cu_of(rep)
    for i in range(n):
        scan_check(y[at[i]:at[i + 1]], S[i], i, inp, cu[i + 1] - rep[i], cu[i + 1], torch.zeros(h, k, p, dtype=torch.float64), dt, True,
                   "window %d" % i)


@TYPES
def test_scan_gates_far_apart(dt):
    # strong decays (a = 0 in fp32 among them) in front of weak ones, in one chunk: the weak ones keep
    # their accuracy; dt = 0 and a gate of exactly 1 too
    g, h, k, p, T = 1, 2, 64, 64, 192
    r = Rand(9)
    inp = scan_inputs(r, T, g, h, k, p, dt, False)
    inp["dt_bias"] = torch.zeros(h, device="cuda")
    v = torch.full((T, h), 0.0039, device="cuda")
    v[5], v[70], v[100], v[101], v[130] = 30.0, 3000.0, 0.0, 12.0, 1e6
    inp["dt"] = v.to(dt)
    inp["A"] = ints([-1, -3]).float()
    S, y, _ = G().gdn_ssm_scan(**inp, cu_seqlens=ints([0, T]), softplus=False)
    scan_check(y, S[0], 0, inp, 0, T, torch.zeros(h, k, p, dtype=torch.float64), dt, False, "gates")


# ------------------------------------------------------------------ single tokens
@TYPES
@pytest.mark.parametrize("g,h,k,p,rows", [(1, 1, 64, 64, 1), (2, 6, 128, 64, 5), (4, 4, 64, 128, 70), (1, 2, 128, 128, 3)])
def test_ssm_step(dt, g, h, k, p, rows):
    r = Rand(rows + h)
    inp = scan_inputs(r, rows, g, h, k, p, dt, True)
    S = r.n(rows + 2, h, k, p)
    slots = r.perm(rows + 2)[:rows].to(torch.int32)
    if rows > 2:
        slots[2] = -1
    before, y, ws = S.clone(), torch.full((rows, h, p), 7.0, dtype=dt, device="cuda"), new_ws()
    say("ssm_step", dt, g, h, k, p, rows)
    cu = inp.pop("x"), inp.pop("B"), inp.pop("C"), inp.pop("dt"), inp.pop("A")
    G().gdn_ssm_step(*cu, S, slots=slots.cuda(), y=y, ws=ws, **inp)
    assert G().gdn_device_status(ws) == 0
    used = [s for s in slots.tolist() if s >= 0]
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            assert (y[i] == 7).all()
            continue
        x, B, C, dtv, A = cu
        ref = R.ssm_tokens(R.d(x[i:i + 1]), R.d(B[i:i + 1]), R.d(C[i:i + 1]), R.d(dtv[i:i + 1]), R.d(A), R.d(inp["D"]),
                           R.d(inp["dt_bias"]), R.d(before[s]))
        # state: the gate (14 roundings) and two products and a sum; y: a sum over d_k on top
        R.within(S[s], ref[2], 20 * R.U32 * ref[3], "S of row %d" % i)
        R.within(y[i:i + 1], ref[0], R.u(dt) * ref[0].abs() + (30 + k) * R.U32 * ref[1], "y of row %d" % i)
    rest = [s for s in range(rows + 2) if s not in used]
    assert torch.equal(S[rest], before[rest])


@TYPES
@pytest.mark.parametrize("g,h,k,p,rows,f32_out", [(1, 1, 64, 64, 1, False), (2, 4, 128, 128, 9, True), (3, 3, 128, 64, 66, False)])
def test_delta_step(dt, g, h, k, p, rows, f32_out):
    r = Rand(rows + k)
    q, kk = (torch.nn.functional.normalize(r.n(rows, g, k), dim=-1).to(dt) for _ in range(2))
    v, gate, beta = r.n(rows, h, p, dt=dt), -r.n(rows, h).abs(), torch.rand(rows, h, generator=r.g).cuda()
    gate[0, 0] = -math.inf                                     # a = 0: a reset
    S = r.n(rows + 2, h, k, p, scale=0.3)
    slots = r.perm(rows + 2)[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1
    before, ws, scale = S.clone(), new_ws(), 0.7
    say("delta_step", dt, g, h, k, p, rows)
    o = G().gdn_step(q, kk, v, gate, beta, S, slots=slots.cuda(), scale=scale, o_dtype=F32 if f32_out else None, ws=ws)
    assert G().gdn_device_status(ws) == 0
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        ref = R.delta_token(R.d(q[i]), R.d(kk[i]), R.d(v[i]), R.d(gate[i]), R.d(beta[i]), R.d(before[s]), scale)
        # the sum over d_k in front of the update, the gate, and the update itself; o: one more sum
        R.within(S[s], ref[2], (k + 20) * R.U32 * ref[3], "S of row %d" % i)
        R.within(o[i], ref[0], R.u(o.dtype) * ref[0].abs() + (2 * k + 30) * R.U32 * ref[1], "o of row %d" % i)
    rest = [s for s in range(rows + 2) if s not in slots.tolist()]
    assert torch.equal(S[rest], before[rest])
    # without slots: state i for row i, the same numbers
    pool = before[:rows].clone()
    a = G().gdn_step(q, kk, v, gate, beta, pool, scale=scale)
    pool2 = before[:rows].clone()
    b = G().gdn_step(q, kk, v, gate, beta, pool2, slots=torch.arange(rows, dtype=torch.int32, device="cuda"), scale=scale)
    assert torch.equal(a, b) and torch.equal(pool, pool2)


def test_bad_slots_are_reported_and_change_nothing():
    r = Rand(3)
    rows, h, k, p = 6, 2, 64, 64
    inp = scan_inputs(r, rows, 1, h, k, p, F32, True)
    args = [inp[n] for n in ("x", "B", "C", "dt", "A")]
    S, ws = r.n(5, h, k, p), new_ws()
    before, y = S.clone(), torch.full((rows, h, p), 7.0, device="cuda")
    slots = ints([2, 5, 2, -2, -1, 0])                        # row 1 out of range, 2 taken, 3 negative, 4 padded
    G().gdn_ssm_step(*args, S, slots=slots, y=y, ws=ws)
    assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT and G().gdn_device_status(ws) == 0
    assert (y[1:5] == 7).all() and not (y[0] == 7).any() and not (y[5] == 7).any()
    assert torch.equal(S[[1, 3, 4]], before[[1, 3, 4]]) and not torch.equal(S[2], before[2])
    x, w, state = r.n(rows, 64), r.n(64, 4), r.n(5, 3, 64)
    before, y = state.clone(), torch.full((rows, 64), 7.0, device="cuda")
    G().gdn_conv_step(x, w, state, slots=slots, y=y, ws=ws)
    assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT
    assert (y[1:5] == 7).all() and torch.equal(state[[1, 3, 4]], before[[1, 3, 4]])


def test_bad_cu_seqlens_is_reported():
    r = Rand(4)
    x, w = r.n(20, 64), r.n(64, 4)
    inp = scan_inputs(r, 20, 1, 1, 64, 64, F32, True)
    for cu in ([0, 8, 5, 20], [0, 25], [-1, 20], [0, 30, 20], [3, 20]):
        ws = new_ws(1 << 20)
        G().gdn_conv(x, w, ints(cu), ws=ws)
        assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT, cu
        G().gdn_ssm_scan(**inp, cu_seqlens=ints(cu), ws=ws)
        assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT, cu
    ws = new_ws()
    G().gdn_ssm_scan(**inp, cu_seqlens=ints([0, 20]), r=ints([21]), total_out_tokens=20, ws=ws)
    assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT
    G().gdn_ssm_scan(**inp, cu_seqlens=ints([0, 20]), r=ints([9]), total_out_tokens=8, ws=ws)     # y too short
    assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT


# ------------------------------------------------------------------ norm, rotation, append
class Cache:
    """A paged cache with pages in a shuffled order, NaN in every cell that no sequence owns."""

    def __init__(self, r, kv, ps, hk, d, dt, heads_first=False, spare=2):
        self.ps, self.kv = ps, kv
        per = [-(-x // ps) for x in kv]
        pages = sum(per) + spare
        shape = (pages, hk, ps, d) if heads_first else (pages, ps, hk, d)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dt, device="cuda") for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = r.perm(pages).tolist()
        self.pages = [[order.pop() for _ in range(p)] for p in per]
        most = max(per + [1]) + 1
        self.table = ints([row + [-1] * (most - len(row)) for row in self.pages])
        self.keys = [r.n(x, hk, d, dt=dt) for x in kv]
        self.vals = [r.n(x, hk, d, dt=dt) for x in kv]
        for i, x in enumerate(kv):
            for j in range(x):
                self.k[self.pages[i][j // ps], j % ps] = self.keys[i][j]
                self.v[self.pages[i][j // ps], j % ps] = self.vals[i][j]


ROPE = [  # h_q, h_kv, d, rot, page, lengths, context, interleaved, norm
    (1, 1, 64, 16, 16, [1], [0], False, True), (6, 2, 128, 128, 24, [5, 0, 1, 40], [3, 9, 0, 17], True, True),
    (16, 2, 256, 64, 1, [3, 2], [5, 0], False, True), (4, 4, 64, 64, 64, [70], [100], False, False),
    (3, 1, 128, 0, 16, [9], [2], False, True), (33, 1, 256, 256, 32, [2], [30], True, True),
]


@TYPES
@pytest.mark.parametrize("hq,hk,dim,rot,ps,lens,ctx,inter,norm", ROPE)
def test_norm_rope_append(dt, hq, hk, dim, rot, ps, lens, ctx, inter, norm):
    r = Rand(dim + hq)
    cu, n = cu_of(lens), len(lens)
    T, kv = cu[-1], [a + b for a, b in zip(lens, ctx)]
    c = Cache(r, kv, ps, hk, dim, dt, heads_first=inter)
    wide = r.n(T + 2, (hq + 2 * hk) * dim + 8, dt=dt)
    q, k, v = (wide[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    wq, wk = r.n(dim), (r.n(dim) if hq > 1 else None)
    ang = torch.rand(max(kv) + 1, rot // 2, generator=r.g).double() * 100
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    out, ws = torch.full((T + 2, hq, dim), 7.0, dtype=dt, device="cuda"), new_ws()
    k0, v0 = c.k.clone(), c.v.clone()
    say("norm_rope", dt, hq, hk, dim, rot, ps, lens, ctx)
    G().gdn_qk_norm_rope(q, k, v, cs, c.k, c.v, c.table, ints(cu), ints(kv), q_weight=wq, k_weight=wk, norm=norm,
                         interleaved=inter, q_out=out, ws=ws)
    assert G().gdn_device_status(ws) == 0
    assert (out[T:] == 7).all()
    # the sum of squares over d, root and quotient, the weight, two products and a sum
    ops = dim + 12
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for i in range(n):
        for j in range(lens[i]):
            t, pos = cu[i] + j, ctx[i] + j
            cos, sin = R.d(cs[pos, :rot // 2]), R.d(cs[pos, rot // 2:])
            ref, ab = R.rope_head(R.d(q[t]), R.d(wq), 1e-6, norm, cos, sin, inter)
            R.within(out[t], ref, R.u(dt) * ref.abs() + ops * R.U32 * ab, "q of token %d" % t)
            ref, ab = R.rope_head(R.d(k[t]), R.d(wk) if wk is not None else None, 1e-6, norm, cos, sin, inter)
            page = c.pages[i][pos // ps]
            R.within(c.k[page, pos % ps], ref, R.u(dt) * ref.abs() + ops * R.U32 * ab, "k of token %d" % t)
            assert torch.equal(c.v[page, pos % ps], v[t])
            touched[page, pos % ps] = True
    # every other cell of the caches is as it was
    assert torch.equal(c.k[~touched.cuda()].nan_to_num(), k0[~touched.cuda()].nan_to_num())
    assert torch.equal(c.v[~touched.cuda()].nan_to_num(), v0[~touched.cuda()].nan_to_num())
    # in place of q, and by positions of the caller's
    again = q.contiguous()
    G().gdn_qk_norm_rope(again, k, v, cs, c.k, c.v, c.table, ints(cu), ints(kv), q_weight=wq, k_weight=wk, norm=norm,
                         interleaved=inter, q_out=again, ws=ws,
                         positions=ints([ctx[i] + j for i in range(n) for j in range(lens[i])] + [0, 0]))
    assert torch.equal(again[:T], out[:T])


def test_append_reports_bad_places():
    r = Rand(8)
    hq, hk, dim, ps = 2, 1, 64, 16
    cs = torch.cat([torch.ones(40, 32), torch.zeros(40, 32)], 1).cuda()
    q, k, v = (r.n(4, h, dim) for h in (hq, hk, hk))

    def call(kv, table, pages=3, positions=None):
        kc, vc, ws = torch.full((pages, ps, hk, dim), 5.0, device="cuda"), torch.full((pages, ps, hk, dim), 5.0, device="cuda"), new_ws()
        G().gdn_qk_norm_rope(q, k, v, cs, kc, vc, ints([table]), ints([0, 4]), ints([kv]), positions=positions, ws=ws)
        return G().gdn_device_status(ws), int((vc != 5).any(-1).sum())

    bad = G().GDN_ERR_DEVICE_INPUT
    assert call(20, [0, 2]) == (0, 4)
    assert call(18, [0, 3]) == (bad, 2)            # the second page does not exist
    assert call(18, [-1, 2]) == (bad, 2)
    assert call(33, [0, 2]) == (bad, 0)            # more tokens than the table holds
    assert call(-1, [0, 2]) == (bad, 0)
    assert call(3, [0, 2]) == (bad, 3)             # the first token has no place
    assert call(20, [0, 2], positions=ints([0, 39, 40, -1])) == (bad, 2)


# ------------------------------------------------------------------ attention
ATTN = [  # h_q, h_kv, d, page, lengths, context, heads first
    (1, 1, 64, 16, [1], [0], False), (8, 2, 128, 16, [1, 1, 1], [0, 63, 200], False),
    (6, 2, 64, 24, [1, 0, 1, 1], [500, 7, 31, 32], True), (16, 2, 256, 64, [1, 1], [700, 1], False),
    (4, 4, 128, 1, [2, 1], [40, 3], False), (32, 1, 64, 32, [1, 1], [90, 300], False),
    (8, 2, 128, 16, [70, 1, 0, 130], [0, 200, 5, 33], False), (16, 2, 256, 64, [65], [190], False),
    (3, 1, 64, 48, [129, 2], [0, 64], True), (5, 5, 128, 128, [33], [1], False),
    # 17 to 32 rows a sequence
    (24, 1, 64, 16, [1, 1, 0, 1], [300, 5, 9, 64], False), (20, 1, 256, 32, [1, 1], [130, 700], True),
    (24, 1, 128, 16, [1, 1], [90, 257], False), (8, 2, 64, 16, [8, 3, 0, 9], [500, 0, 7, 31], False),
    (4, 2, 256, 16, [16, 1, 12], [70, 300, 0], False),
    # 192 rows a sequence and more: large tiles of rows, one split, a few splits, many
    (8, 2, 128, 16, [70, 50, 130], [0, 90, 33], False), (4, 1, 256, 64, [300], [700], False),
    (8, 1, 64, 16, [41, 30, 2], [2100, 0, 64], True),
    # contexts that one workgroup takes whole
    (8, 2, 128, 16, [1, 1], [500, 3], False), (4, 2, 64, 16, [1, 1, 1], [700, 0, 65], True), (16, 2, 256, 64, [1, 1], [200, 31], False),
    # long contexts, ragged, one of them empty; many rows in a few splits
    (4, 2, 64, 16, [1, 1, 1, 0], [5000, 0, 4200, 33], False), (16, 2, 256, 64, [1, 2], [4099, 70], True),
    (32, 8, 128, 16, [1, 1], [5300, 1100], False), (16, 2, 64, 16, [300], [1800], False),
]


def attn_tols(o, oa, lse, big, dt, d, n):
    # a score is a sum of d products, the scale and the base change: off by (d + 4) u times its abs;
    # probabilities move by twice that relatively, and by the exponential and the sums over n keys
    # (4 roundings for each of up to n / 32 rescales along the way); bf16: the rounding of P
    s = 2 * (d + 4) * R.U32 * big + (n + 8) * R.U32
    rel = s[:, None] + (R.u(dt) if dt is BF else 0.0)
    return R.u(dt) * o.abs() + rel * (1 + 2 ** -6) * oa + 1e-30, s + 4 * R.U32 * lse.abs().nan_to_num(posinf=0.0)


def attn_check(c, q, o, lse, lens, kv, scale, dt, what=""):
    cu = cu_of(lens)
    for i, L in enumerate(lens):
        for j in range(L):
            t, pos = cu[i] + j, kv[i] - L + j
            ref, oa, l, big = R.attend(R.d(q[t]), R.d(c.keys[i]), R.d(c.vals[i]), pos, scale)
            to, tl = attn_tols(ref, oa, l, big, dt, q.shape[-1], max(pos + 1, 0))
            R.within(o[t], ref, to, "%s o of token %d of sequence %d" % (what, j, i))
            if lse is not None:
                if pos < 0:
                    assert (lse[t] == -math.inf).all()
                else:
                    R.within(lse[t], l, tl, "%s lse of token %d of sequence %d" % (what, j, i))


@TYPES
@pytest.mark.parametrize("hq,hk,dim,ps,lens,ctx,hf", ATTN)
def test_attention(dt, hq, hk, dim, ps, lens, ctx, hf):
    r = Rand(dim + hq + len(lens))
    kv = [a + b for a, b in zip(lens, ctx)]
    T = sum(lens)
    c = Cache(r, kv, ps, hk, dim, dt, heads_first=hf)
    q = r.n(T + 2, hq * dim + 16, dt=dt)[:, :hq * dim].unflatten(1, (hq, dim))
    o = torch.full((T + 2, hq, dim), 7.0, dtype=dt, device="cuda")
    lse, ws = torch.full((T + 2, hq), 7.0, device="cuda"), new_ws(1 << 28)
    say("attention", dt, hq, hk, dim, ps, lens, ctx)
    G().gdn_paged_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), max_kv_len=max(kv), o=o, lse=lse, ws=ws)
    assert G().gdn_device_status(ws) == 0
    assert (o[T:] == 7).all() and (lse[T:] == 7).all()
    attn_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)


@TYPES
@pytest.mark.parametrize("lens,kv", [([1, 1], [3000, 1]), ([1, 1], [0, 2500]), ([40, 3], [2300, 1000]), ([20], [12])])
def test_attention_splits_and_empty_rows(dt, lens, kv):
    # keys split over workgroups (a bound far over some lengths), rows and whole sequences that see
    # nothing, a scale of the caller's
    hq, hk, dim = 4, 2, 64
    r = Rand(kv[0])
    c = Cache(r, kv, 16, hk, dim, dt)
    q, ws = r.n(sum(lens), hq, dim, dt=dt, scale=2.0), new_ws(1 << 26)
    say("attention splits", dt, lens, kv)
    o, lse = G().gdn_paged_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), scale=0.25, lse=True, ws=ws)
    assert G().gdn_device_status(ws) == 0
    attn_check(c, q, o, lse, lens, kv, 0.25, dt)


@TYPES
@pytest.mark.parametrize("lens,kv", [([1, 1], [700, 90]), ([40], [260])])
def test_attention_scale_of_any_sign(dt, lens, kv):
    hq, hk, dim = 4, 1, 64
    r = Rand(21)
    c = Cache(r, kv, 16, hk, dim, dt)
    q = r.n(sum(lens), hq, dim, dt=dt)
    for scale in (0.0, -0.3):
        o, lse = G().gdn_paged_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), scale=scale, lse=True)
        attn_check(c, q, o, lse, lens, kv, scale, dt)


def test_attention_large_scores():
    # scores of several hundred, rising and falling along the keys: the running maximum matters
    dt, hq, hk, dim, kv = F32, 2, 1, 64, 300
    r = Rand(1)
    c = Cache(r, [kv], 16, hk, dim, dt)
    for x in (c.keys[0],):
        x.mul_(torch.linspace(-30, 30, kv, device="cuda").cos()[:, None, None] * 40)
    for j in range(kv):
        c.k[c.pages[0][j // 16], j % 16] = c.keys[0][j]
    q = r.n(7, hq, dim, dt=dt)
    o, lse = G().gdn_paged_attn(q, c.k, c.v, c.table, ints([0, 7]), ints([kv]), scale=1.0, lse=True)
    attn_check(c, q, o, lse, [7], [kv], 1.0, dt)


def test_attention_reports_bad_input():
    r = Rand(2)
    kv, bad = [40, 33], G().GDN_ERR_DEVICE_INPUT
    c = Cache(r, kv, 16, 1, 64, BF)
    for lens in ([1, 1], [50, 30]):
        T = sum(lens)
        q = r.n(T, 2, 64, dt=BF)

        def call(table=c.table, kv_len=kv, cu=cu_of(lens), most=48):
            ws = new_ws(1 << 22)
            o = G().gdn_paged_attn(q, c.k, c.v, table, ints(cu), ints(kv_len), max_kv_len=most, ws=ws)
            return G().gdn_device_status(ws), o

        st, o = call()
        assert st == 0
        t = c.table.clone()
        t[0, 1] = c.k.shape[0]
        st, o2 = call(table=t)
        assert st == bad and torch.equal(o2[lens[0]:], o[lens[0]:])     # the other sequence is right
        t[0, 1] = -1
        assert call(table=t)[0] == bad
        assert call(kv_len=[49, 33])[0] == bad and call(kv_len=[-1, 33])[0] == bad
        assert call(cu=[0, T + 1, T])[0] == bad


# ------------------------------------------------------------------ apart
def test_rows_far_apart():
    """Rows, states' neighbours and pages more than 2^31 elements apart, against the same call on
    compact tensors: the same arithmetic, so the same bits."""
    g = G()
    r = Rand(3)
    T, h, hq, hk, dim, ps = 300, 2, 4, 2, 64, 16
    far = torch.empty(T, 1 << 23, dtype=BF, device="cuda")        # row 299 is 2.5e9 elements in
    at = [0]

    def place(t):
        n = t[0].numel()
        v = far[:, at[0]:at[0] + n].unflatten(1, t.shape[1:])
        at[0] += -(-n // 8) * 8                                   # the next one starts on 16 bytes
        v.copy_(t)
        return v

    cu = ints([0, 290, 300])
    x, w = r.n(T, 256, dt=BF), r.n(256, 4)
    y, st = g.gdn_conv(x, w, cu)
    y2, st2 = g.gdn_conv(place(x), w, cu, y=place(torch.zeros_like(y)))
    assert torch.equal(y, y2) and torch.equal(st, st2)
    inp = {n: (t.contiguous() if t is not None else t) for n, t in scan_inputs(r, T, 1, h, 64, 64, BF, True).items()}
    S, y, _ = g.gdn_ssm_scan(**inp, cu_seqlens=cu)
    apart = {n: place(t) if n in ("x", "B", "C") else t for n, t in inp.items()}
    apart["dt"] = place(inp["dt"])
    S2, y2, _ = g.gdn_ssm_scan(**apart, cu_seqlens=cu, y_out=place(torch.zeros_like(y)))
    assert torch.equal(S, S2) and torch.equal(y, y2)
    pool, pool2 = (torch.ones(T, 3, 256, dtype=BF, device="cuda") for _ in range(2))
    y = g.gdn_conv_step(x, w, pool)
    assert torch.equal(y, g.gdn_conv_step(place(x), w, pool2, y=place(torch.zeros_like(y)))) and torch.equal(pool, pool2)
    S, S2 = (torch.ones(T, h, 64, 64, device="cuda") for _ in range(2))
    a, b = ([d[n] for n in ("x", "B", "C", "dt", "A")] for d in (inp, apart))
    y = g.gdn_ssm_step(*a, S)
    assert torch.equal(y, g.gdn_ssm_step(*b, S2, y=place(torch.zeros_like(y)))) and torch.equal(S, S2)
    q, k, v = r.n(T, hq, dim, dt=BF), r.n(T, hk, dim, dt=BF), r.n(T, hk, dim, dt=BF)
    cs, kv = r.n(400, dim), ints([290, 60])
    c = Cache(r, [290, 60], ps, hk, dim, BF)
    qr = g.gdn_qk_norm_rope(q, k, v, cs, c.k, c.v, c.table, cu, kv)
    k1, v1 = c.k.clone(), c.v.clone()
    qr2 = g.gdn_qk_norm_rope(place(q), place(k), place(v), cs, c.k, c.v, c.table, cu, kv, q_out=place(torch.zeros_like(q)))
    assert torch.equal(qr, qr2) and torch.equal(k1.nan_to_num(), c.k.nan_to_num()) and torch.equal(v1.nan_to_num(), c.v.nan_to_num())
    # caches whose last pages are used: more than 2^31 elements, 4 GiB and more
    pages = 1100000
    base = pages - c.k.shape[0]
    K, V = (torch.empty(pages, ps, hk, dim, dtype=BF, device="cuda") for _ in range(2))
    K[base:], V[base:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + base, c.table)
    assert torch.equal(qr, g.gdn_qk_norm_rope(q, k, v, cs, K, V, table, cu, kv))
    assert torch.equal(K[base:].nan_to_num(), c.k.nan_to_num()) and torch.equal(V[base:].nan_to_num(), c.v.nan_to_num())
    one = ints([0, 1, 2])
    for n, cus in ((T, cu), (2, one)):
        o = g.gdn_paged_attn(qr[:n], c.k, c.v, c.table, cus, kv)
        assert torch.equal(o, g.gdn_paged_attn(qr2[:n], K, V, table, cus, kv, o=place(torch.zeros_like(q))[:n]))
    # a pool of states whose used slots are 2^31 elements in
    pool = torch.empty(600000, h, 64, 64, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda") + (600000 - T)
    pool[600000 - T:] = 1.0
    y2 = g.gdn_ssm_step(*a, pool, slots=slots)
    assert torch.equal(y, y2) and torch.equal(pool[600000 - T:], S2)


def test_a_sequence_does_not_reach_its_neighbours():
    """A sequence of NaN, NaN behind the last one and in front of a window: the others' bits stay."""
    g = G()
    r = Rand(41)
    lens, h, hq, hk, dim = [70, 33, 100], 2, 4, 2, 64
    cu, T = cu_of(lens), sum(lens)
    mine = torch.ones(T + 5, dtype=torch.bool, device="cuda")
    mine[cu[1]:cu[2]] = False
    mine[T:] = False

    def both(x):
        bad = x.clone()
        bad[~mine] = math.nan
        return x, bad

    w, cut = r.n(128, 4), ints(cu)
    for dt in (BF, F32):
        xs = both(r.n(T + 5, 128, dt=dt))
        (y, s), (y2, s2) = (g.gdn_conv(x, w, cut) for x in xs)
        assert torch.equal(y[mine], y2[mine]) and torch.equal(s[::2], s2[::2])
        inp = {n: (t.contiguous() if t is not None else t) for n, t in scan_inputs(r, T + 5, 1, h, 64, 64, dt, True).items()}
        bad = dict(inp)
        for n in ("x", "B", "C", "dt"):
            bad[n] = both(inp[n])[1]
        (S, y, _), (S2, y2, _) = (g.gdn_ssm_scan(**i, cu_seqlens=cut) for i in (inp, bad))
        assert torch.equal(y[mine], y2[mine]) and torch.equal(S[::2], S2[::2])
        rep = ints([20, 33, 100])
        mine[:cu[1] - 20] = False
        for n in ("x", "B", "C", "dt"):
            bad[n] = both(inp[n])[1]
        (S, y, _), (S2, y2, _) = (g.gdn_ssm_scan(**i, cu_seqlens=cut, r=rep, total_out_tokens=153) for i in (inp, bad))
        assert torch.equal(y[:20], y2[:20]) and torch.equal(y[53:], y2[53:]) and torch.equal(S[::2], S2[::2])
        mine[:cu[1]] = True
        for L in (lens, [1, 1, 1]):
            kv, cus = [90, 33, 100], ints(cu_of(L))
            c = Cache(r, kv, 16, hk, dim, dt)
            q = r.n(sum(L), hq, dim, dt=dt)
            o = g.gdn_paged_attn(q, c.k, c.v, c.table, cus, ints(kv))
            for p in c.pages[1]:
                c.k[p], c.v[p] = math.nan, math.nan
            o2 = g.gdn_paged_attn(q, c.k, c.v, c.table, cus, ints(kv))
            a, b = L[0], L[0] + L[1]
            assert torch.equal(o[:a], o2[:a]) and torch.equal(o[b:], o2[b:])


def test_two_streams_at_once():
    """The same operators on two streams, each with workspaces of its own, against one after the other."""
    g = G()
    r = Rand(51)
    inp = [scan_inputs(r, 1500, 1, 4, 64, 64, BF, True) for _ in range(2)]
    cu, kv = ints([0, 1500]), [2500, 900]
    c = Cache(r, kv, 16, 2, 64, BF)
    q = [r.n(2, 4, 64, dt=BF) for _ in range(2)]
    wss = [[new_ws(1 << 24), new_ws(1 << 24)] for _ in range(2)]
    cut, kvt = ints([0, 1, 2]), ints(kv)

    def calls(i, stream):
        S, y, _ = g.gdn_ssm_scan(**inp[i], cu_seqlens=cu, ws=wss[i][0], stream=stream)
        return S, y, g.gdn_paged_attn(q[i], c.k, c.v, c.table, cut, kvt, ws=wss[i][1], stream=stream)

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[calls(i, streams[i]) for i in range(2)] for _ in range(5)]
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ together
@TYPES
def test_prompt_then_tokens(dt):
    """A hybrid's layers over a prompt in one piece, against the same prompt as a prefix, a suffix
    continued from the prefix's states and cache, and three single tokens."""
    g = G()
    r = Rand(77)
    W, ch, h, hq, hk, dim, ps = 4, 3 * 64 + 64, 1, 4, 2, 64, 16
    cuts = [90, 41, 1, 1, 1]                                   # prefix, suffix, tokens
    L = sum(cuts)
    x, w = r.n(L, ch, dt=dt), r.n(ch, W, scale=0.5)
    gates, beta = -r.n(L, h).abs() * 0.1, torch.rand(L, h, generator=r.g).cuda()
    dtr, A = r.n(L, h, dt=dt), ints([-2]).float()
    q, k, v = r.n(L, hq, dim, dt=dt), r.n(L, hk, dim, dt=dt), r.n(L, hk, dim, dt=dt)
    ang = torch.arange(L).double()[:, None] * 10000.0 ** (-torch.arange(0, dim, 2).double() / dim)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()

    def layer(pieces):
        state, S, Sg = None, None, None
        kc, vc = (torch.full((16, ps, hk, dim), math.nan, dtype=dt, device="cuda") for _ in range(2))
        table = ints([[9, 3, 15, 0, 7, 1, 12, 4, 11, 2]])
        outs, lo = [], 0
        for n in pieces:
            hi, cu = lo + n, ints([0, n])
            if n == 1 and lo > 0:
                y = g.gdn_conv_step(x[lo:hi], w, state)
            else:
                y, state = g.gdn_conv(x[lo:hi], w, cu, state0=state)
            a, b, c, d = (t.unflatten(1, (h, 64)) for t in y.split(64, 1))
            qn, kn = (torch.nn.functional.normalize(t.float(), dim=-1).to(dt).contiguous() for t in (a, b))
            vv = c.contiguous()
            if n == 1 and lo > 0:
                o = g.gdn_step(qn, kn, vv, gates[lo:hi], beta[lo:hi], Sg)
                z = g.gdn_ssm_step(d, b, a, dtr[lo:hi], A, S)
            else:
                Sg, o = g.gdn_prefill(qn, kn, vv, gates[lo:hi].clone(), beta[lo:hi].clone(), cu, S0=Sg)
                S, z, _ = g.gdn_ssm_scan(d, b, a, dtr[lo:hi], A, cu, S0=S)
            kv = ints([hi])
            qr = g.gdn_qk_norm_rope(q[lo:hi], k[lo:hi], v[lo:hi], cs, kc, vc, table, cu, kv)
            f = g.gdn_paged_attn(qr, kc, vc, table, cu, kv)
            outs.append((o, z, f))
            lo = hi
        return [torch.cat(p) for p in zip(*outs)] + [S, Sg, state]

    one, many = layer([L]), layer(cuts)
    names = ("gated delta", "state space", "attention", "S", "S gated", "conv state")
    # both are right to the operators' own tolerances: a relative Frobenius distance of twice the
    # type's few roundings (the gated delta prefill is held to 3e-3 and 1e-5 by its own tests, the
    # sums here have at most 64 + 128 fp32 roundings)
    for name, a, b in zip(names, one, many):
        rel = float((a.double() - b.double()).norm() / a.double().norm())
        say("  %s: one piece against five, relative %.2e" % (name, rel))
        assert rel <= (2 * 3 * 2 ** -8 if dt is BF else 2 * 1e-5 + 400 * R.U32), name


@pytest.mark.parametrize("own_stream", [False, True])
def test_captured_step_replays(own_stream):
    """Every operator captured in one graph and replayed between eager work, bit for bit."""
    g = G()
    r = Rand(31)
    rows, h, hq, hk, dim, kv = 5, 2, 4, 2, 64, [700, 33, 1, 64, 300]
    x, w, pool = r.n(rows, 64, dt=BF), r.n(64, 4), r.n(rows, 3, 64, dt=BF)
    inp = scan_inputs(r, rows, 1, h, 64, 64, BF, True)
    args = [inp[n] for n in ("x", "B", "C", "dt", "A")]
    S, S0 = r.n(rows, h, 64, 64), None
    c = Cache(r, kv, 16, hk, dim, BF)
    q, k, v = r.n(rows, hq, dim, dt=BF), r.n(rows, hk, dim, dt=BF), r.n(rows, hk, dim, dt=BF)
    cs, cu, kvt = torch.ones(800, 64, device="cuda"), ints(list(range(rows + 1))), ints(kv)
    long = scan_inputs(r, 1500, 1, 1, 64, 64, BF, True)
    lx, lw = r.n(1500, 64, dt=BF), r.n(64, 3)
    lcu = ints([0, 1500])
    S0, pool0 = S.clone(), pool.clone()
    bufs = dict(y=torch.empty_like(x), z=torch.empty_like(inp["x"].contiguous()), qo=torch.empty_like(q), o=torch.empty_like(q),
                lse=torch.empty(rows, hq, device="cuda"), ly=torch.empty_like(lx), ls=torch.empty(1, 2, 64, dtype=BF, device="cuda"),
                lS=torch.empty(1, 1, 64, 64, device="cuda"), lz=torch.empty(1500, 1, 64, dtype=BF, device="cuda"))
    wss = [new_ws(1 << 24) for _ in range(6)]
    stream = torch.cuda.Stream() if own_stream else None

    def calls(stream=None):
        g.gdn_conv_step(x, w, pool, y=bufs["y"], ws=wss[0], stream=stream)
        g.gdn_ssm_step(*args, S, D=inp["D"], dt_bias=inp["dt_bias"], y=bufs["z"], ws=wss[1], stream=stream)
        g.gdn_qk_norm_rope(q, k, v, cs, c.k, c.v, c.table, cu, kvt, q_out=bufs["qo"], ws=wss[2], stream=stream)
        g.gdn_paged_attn(bufs["qo"], c.k, c.v, c.table, cu, kvt, o=bufs["o"], lse=bufs["lse"], ws=wss[3], stream=stream)
        g.gdn_conv(lx, lw, lcu, state_out=bufs["ls"], y=bufs["ly"], ws=wss[4], stream=stream)
        g.gdn_ssm_scan(**long, cu_seqlens=lcu, S_out=bufs["lS"], y_out=bufs["lz"], ws=wss[5], stream=stream)

    calls()
    torch.cuda.synchronize()
    want = {n: b.clone() for n, b in bufs.items()}
    wS, wpool = S.clone(), pool.clone()
    if own_stream:                                             # the same calls on the caller's stream
        S.copy_(S0), pool.copy_(pool0)
        torch.cuda.synchronize()
        calls(stream)
        stream.synchronize()
        assert all(torch.equal(b, want[n]) for n, b in bufs.items()) and torch.equal(S, wS) and torch.equal(pool, wpool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    a = torch.randn(256, 256, device="cuda")
    for rep in range(3):
        S.copy_(S0), pool.copy_(pool0)
        for b in bufs.values():
            b.fill_(math.nan)
        (a @ a).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, b in bufs.items():
            assert torch.equal(b, want[n]), (rep, n)
        assert torch.equal(S, wS) and torch.equal(pool, wpool)
    assert all(g.gdn_device_status(ws) == 0 for ws in wss)
