"""GPU: the operators around a prefix cache against plain 64-bit implementations (prefix_reference.py).

Whole numbers are equal.  Tolerances of computed numbers count roundings, as in test_gpu_ops.py."""
import math
import random

import pytest
import torch

import ops_reference as R
import prefix_reference as PR
from gpu_helpers import say
from test_gpu_ops import BF, F32, TYPES, Rand, attn_tols, cu_of, ints, new_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import gated_deltanet_state_gdn_amd as gdn
    gdn.load()
    yield


def G():
    import gated_deltanet_state_gdn_amd as gdn
    return gdn


# ------------------------------------------------------------------ block tables
def extend_case(seed, n, ps, most_new, prefixes=0, spare=5, empty=0.2):
    r = random.Random(seed)
    pre = [r.randrange(0, 9) * ps for _ in range(prefixes)]
    hit = [r.randrange(-1, prefixes) if prefixes else -1 for _ in range(n)]
    kv = [r.randrange(0, 6 * ps) for _ in range(n)]
    new = [0 if r.random() < empty else r.randrange(0, most_new + 1) for _ in range(n)]
    base = [pre[h] if h >= 0 else k for h, k in zip(hit, kv)]
    width = max([-(-(b + x) // ps) for b, x in zip(base, new)] + [1]) + r.randrange(3)
    table = [[1000000 + i * width + j if j < -(-kv[i] // ps) and hit[i] < 0 else -7 for j in range(width)] for i in range(n)]
    need = sum(-(-(b + x) // ps) - -(-b // ps) for b, x in zip(base, new))
    free = r.sample(range(100000), need + spare)
    pt = [[500000 + 100 * i + j for j in range(9)] for i in range(prefixes)]
    return dict(new=new, kv=kv, table=table, free=free, at=min(3, spare), ps=ps, hit=hit if prefixes else None, pt=pt, pre=pre)


def extend_call(c, total, ws=None, **kw):
    table = torch.tensor(c["table"], dtype=torch.int32, device="cuda").view(len(c["new"]), -1)
    pre = {}
    if c["hit"] is not None:
        pre = dict(prefix_of=ints(c["hit"]), prefix_table=ints(c["pt"]), prefix_len=ints(c["pre"]))
    out = G().gdn_cache_extend(ints(c["new"]), ints(c["kv"]), table, ints(c["free"]), ints([c["at"]]), c["ps"], total, ws=ws, **pre, **kw)
    return (table,) + tuple(out)


EXTEND = [(1, 1, 16, 1, 0), (2, 5, 1, 9, 0), (3, 64, 16, 1, 0), (4, 70, 24, 40, 3), (5, 1, 16, 5000, 0), (6, 1, 16, 5000, 1),
          (7, 1023, 16, 3, 0), (8, 1025, 32, 3, 2), (9, 3000, 16, 7, 4), (10, 65, 128, 300, 8), (11, 2, 1, 6000, 0), (12, 4097, 1, 1, 1)]


@pytest.mark.parametrize("seed,n,ps,most,prefixes", EXTEND)
def test_extend(seed, n, ps, most, prefixes):
    c = extend_case(seed, n, ps, most, prefixes)
    T = sum(c["new"])
    for total in (T, T + 77):
        ws = new_ws(G().gdn_extend_workspace_bytes(n))
        say("extend", seed, n, ps, T, total)
        table, cu, kv, at, slots, positions = extend_call(c, total, ws)
        want = PR.extend(c["new"], c["kv"], c["table"], c["free"], c["at"], ps, total, c["hit"], c["pt"], c["pre"])
        assert G().gdn_device_status(ws) == 0
        for name, got, w in zip(("table", "cu", "kv", "at", "slots", "positions"), (table, cu, kv, at, slots, positions), want):
            assert got.flatten().tolist() == (sum(w, []) if name == "table" else [w] if name == "at" else w), name
        assert slots.dtype == torch.int64 and positions.dtype == torch.int32


def test_extend_in_place_and_without_outputs():
    c = extend_case(21, 40, 16, 30, 2)
    T = sum(c["new"])
    want = PR.extend(c["new"], c["kv"], c["table"], c["free"], c["at"], 16, T, c["hit"], c["pt"], c["pre"])
    table, kv, at = ints(c["table"]), ints(c["kv"]), ints([c["at"]])
    pre = dict(prefix_of=ints(c["hit"]), prefix_table=ints(c["pt"]), prefix_len=ints(c["pre"]))
    out = G().gdn_cache_extend(ints(c["new"]), kv, table, ints(c["free"]), at, 16, T, kv_out=kv, free_out=at, slots=None, positions=None, **pre)
    assert out[3] is None and out[4] is None and out[1] is kv and out[2] is at
    assert table.tolist() == want[0] and out[0].tolist() == want[1] and kv.tolist() == want[2] and at.tolist() == [want[3]]


def test_extend_of_nothing():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu, kv, at, slots, positions = G().gdn_cache_extend(z, z, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), z, ints([0]), 16, 5000)
    assert cu.tolist() == [0] and at.tolist() == [0] and (slots == -1).all() and (positions == -1).all() and slots.numel() == 5000


def test_a_step_that_does_not_fit_takes_nothing():
    bad = G().GDN_ERR_DEVICE_INPUT
    good = extend_case(31, 20, 16, 30, 2)
    T = sum(good["new"])

    def call(total=T, **change):
        c = {**good, **change}
        ws = new_ws(G().gdn_extend_workspace_bytes(20))
        table, cu, kv, at, slots, positions = extend_call(c, total, ws)
        st = G().gdn_device_status(ws)
        if st == bad:
            assert table.tolist() == c["table"] and cu.tolist() == [0] * 21 and kv.tolist() == c["kv"] and at.tolist() == [c["at"]]
            assert (slots == -1).all() and (positions == -1).all()
        return st

    def swap(v, i, x):
        return v[:i] + [x] + v[i + 1:]

    assert call() == 0
    for total in (T, 6000):
        assert call(total, new=swap(good["new"], 19, -1)) == bad
        assert call(total, new=swap(good["new"], 3, 2 ** 31 - 1)) == bad
        assert call(total, hit=swap(good["hit"], 4, 2)) == bad and call(total, hit=swap(good["hit"], 4, -2)) == bad
        assert call(total, pre=[8, good["pre"][1]]) == bad and call(total, pre=[good["pre"][0], 160]) == bad and call(total, pre=[-16, 16]) == bad
        assert call(total, kv=swap(good["kv"], good["hit"].index(-1), -1)) == bad
        assert call(total, kv=swap(good["kv"], good["hit"].index(-1), 2 ** 31 - 1)) == bad
        assert call(total, at=len(good["free"])) == bad and call(total, at=-1) == bad and call(total, at=len(good["free"]) + 1) == bad
    assert call(T - 1) == bad


# ------------------------------------------------------------------ shared prefixes
class SharedCache:
    """Pages of groups of sequences: a group is (prefix, cached tokens of each sequence).  Unused places hold NaN."""

    def __init__(self, r, groups, ps, hk, dim, dt, heads_first=False):
        lens = [(g, kv) for g, (p, kvs) in enumerate(groups) for kv in kvs]
        total = sum(-(-p // ps) for p, _ in groups) + sum(-(-max(kv, 1) // ps) for _, kv in lens) + 4
        order = r.perm(total).tolist()
        shape = (total, hk, ps, dim) if heads_first else (total, ps, hk, dim)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dt, device="cuda") for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        width = max([-(-max(kv, groups[g][0]) // ps) for g, kv in lens] + [1])
        table = torch.full((len(lens), width), -9, dtype=torch.int32)
        self.keys, self.vals = [], []
        n = 0
        for p, kvs in groups:
            pk, pv = r.n(p, hk, dim, dt=dt), r.n(p, hk, dim, dt=dt)
            shared = [order.pop() for _ in range(p // ps)]
            for i, kv in enumerate(kvs):
                keys = torch.cat([pk, r.n(max(kv - p, 0), hk, dim, dt=dt)])
                vals = torch.cat([pv, r.n(max(kv - p, 0), hk, dim, dt=dt)])
                # the first of the group holds the whole prefix, whatever its kv_len
                held = max(kv, p) if i == 0 else kv
                for j in range(-(-held // ps)):
                    page = shared[j] if j < len(shared) else order.pop()
                    table[n, j] = page
                    m = min(ps, held - j * ps)
                    self.k[page, :m], self.v[page, :m] = keys[j * ps:j * ps + m], vals[j * ps:j * ps + m]
                self.keys.append(keys[:kv])
                self.vals.append(vals[:kv])
                n += 1
        self.table = table.cuda()


def shared_check(c, q, o, lse, lens, kv, scale, dt):
    cu = cu_of(lens)
    for i, L in enumerate(lens):
        keys, vals = R.d(c.keys[i]), R.d(c.vals[i])
        for j in range(L):
            t, pos = cu[i] + j, kv[i] - L + j
            ref, oa, l, big = R.attend(R.d(q[t]), keys, vals, pos, scale)
            to, tl = attn_tols(ref, oa, l, big, dt, q.shape[-1], max(pos + 1, 0))
            R.within(o[t], ref, to, "o of token %d of sequence %d" % (j, i))
            if pos < 0:
                assert (lse[t] == -math.inf).all()
            else:
                R.within(lse[t], l, tl, "lse of token %d of sequence %d" % (j, i))


SHARED = [  # h_q, h_kv, d, page, groups (prefix, [(new, own cached before)]), heads first
    (1, 1, 64, 16, [(16, [(1, 0)])], False),
    (8, 2, 128, 16, [(64, [(1, 3), (1, 0), (1, 200)])], False),
    (16, 2, 256, 64, [(700, [(1, 5), (1, 1)]), (0, [(1, 90)]), (128, [(1, 0)])], False),
    # a prefix that ends inside a page; requests without new tokens; empty groups
    (6, 2, 64, 24, [(101, [(1, 7), (0, 3), (2, 40)]), (5, []), (7, [(1, 1)])], True),
    # page 1, prefix 1
    (4, 4, 128, 1, [(1, [(2, 9), (1, 0)]), (33, [(1, 1)])], False),
    # 32 rows and fewer, 128 and more, 256 and more a group
    (32, 1, 64, 32, [(90, [(1, 30)]), (300, [(1, 0), (0, 0)])], False),
    (8, 2, 128, 16, [(600, [(1, i) for i in range(40)])], False),
    (16, 2, 256, 64, [(190, [(1, 3 * i) for i in range(37)]), (65, [(1, 2)] * 5)], False),
    (8, 1, 64, 16, [(500, [(1, i % 7) for i in range(50)]), (33, [(3, 0)] * 20)], True),
    # prompts behind a prefix
    (4, 1, 256, 64, [(300, [(70, 0), (50, 30), (1, 0)])], False), (8, 2, 128, 16, [(90, [(130, 0)]), (0, [(40, 5)])], False),
    (3, 1, 64, 48, [(64, [(129, 0), (2, 0)])], True), (8, 1, 64, 16, [(2100, [(41, 0), (30, 7), (2, 0)])], False),
    # long prefixes in many splits, long own keys
    (4, 2, 64, 16, [(5000, [(1, 3), (1, 4200)])], False), (16, 2, 256, 64, [(4099, [(1, 0), (2, 70)])], True),
]


def shared_sizes(groups):
    kv = [p + own + new for p, s in groups for new, own in s]
    lens = [new for _, s in groups for new, _ in s]
    of = cu_of([len(s) for _, s in groups])
    bounds = dict(max_kv_len=max(kv), max_prefix_len=max(p for p, _ in groups), max_own_len=max(own + new for _, s in groups for new, own in s))
    return lens, kv, of, [p for p, _ in groups], bounds


@TYPES
@pytest.mark.parametrize("hq,hk,dim,ps,groups,hf", SHARED)
def test_shared_attention(dt, hq, hk, dim, ps, groups, hf):
    r = Rand(dim + hq + len(groups))
    lens, kv, of, pre, bounds = shared_sizes(groups)
    T, n = sum(lens), 0
    c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], ps, hk, dim, dt, hf)
    q = r.n(T + 2, hq * dim + 16, dt=dt)[:, :hq * dim].unflatten(1, (hq, dim))
    o = torch.full((T + 2, hq, dim), 7.0, dtype=dt, device="cuda")
    lse = torch.full((T + 2, hq), 7.0, device="cuda")
    ws = new_ws(G().gdn_shared_workspace_bytes(G().make_shared_desc(q, c.k, c.table, len(lens), len(pre), **bounds)))
    say("shared attention", dt, hq, hk, dim, ps, groups)
    G().gdn_shared_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), ints(of), ints(pre), o=o, lse=lse, ws=ws, **bounds)
    assert G().gdn_device_status(ws) == 0
    assert (o[T:] == 7).all() and (lse[T:] == 7).all()
    shared_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)


@TYPES
@pytest.mark.parametrize("groups", [
    [(40, [(3, 30), (2, 41), (5, 2), (1, 0), (1, 50)])],              # positions inside the prefix, kv_len less than it
    [(64, [(1, 0), (1, 64)])], [(300, [(100, 120), (1, 300)])],       # a request with nothing; a prompt into the prefix
    [(20, [(30, 12), (4, 2)])],                                       # more new tokens than cached ones: rows that see nothing
])
def test_shared_attention_inside_the_prefix(dt, groups):
    hq, hk, dim, ps = 8, 2, 64, 16
    r = Rand(len(groups[0][1]))
    # here the second number is kv_len itself
    kv = [k for _, s in groups for _, k in s]
    lens = [x for _, s in groups for x, _ in s]
    of, pre = cu_of([len(s) for _, s in groups]), [p for p, _ in groups]
    c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], ps, hk, dim, dt)
    q = r.n(sum(lens), hq, dim, dt=dt)
    for scale in (0.2, 0.0, -0.3):
        ws = new_ws(1 << 24)
        o, lse = G().gdn_shared_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), ints(of), ints(pre), scale=scale, lse=True, ws=ws)
        assert G().gdn_device_status(ws) == 0
        shared_check(c, q, o, lse, lens, kv, scale, dt)


def test_shared_attention_without_keys():
    # bounds of zero: no side has keys
    r = Rand(5)
    kc = r.n(2, 16, 1, 64)
    q = r.n(3, 2, 64)
    for most in (0, 40):
        ws = new_ws(1 << 20)
        o, lse = G().gdn_shared_attn(q, kc, kc, ints([[0, 1, 1]] * 3), ints([0, 1, 2, 3]), ints([0, 0, 0]), ints([0, 1, 3]), ints([0, 0]),
                                     max_kv_len=most, lse=True, ws=ws)
        assert G().gdn_device_status(ws) == 0 and (o == 0).all() and (lse == -math.inf).all()


def test_shared_attention_reports_bad_input():
    r = Rand(6)
    bad = G().GDN_ERR_DEVICE_INPUT
    groups = [(40, [(1, 3), (1, 9)]), (20, [(1, 0)])]
    lens, kv, of, pre, bounds = shared_sizes(groups)
    for dt in (BF, F32):
        c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], 16, 1, 64, dt)
        q = r.n(3, 2, 64, dt=dt)

        def call(table=c.table, kv_len=kv, cu=cu_of(lens), groups=of, prefix=pre, **kw):
            ws = new_ws(1 << 22)
            o = G().gdn_shared_attn(q, c.k, c.v, table, ints(cu), ints(kv_len), ints(groups), ints(prefix), ws=ws, **{**bounds, **kw})
            return G().gdn_device_status(ws), o

        st, o = call()
        assert st == 0
        for t0, t1, same in ((0, 1, 2), (2, 0, 0)):              # a page of one group leaves the other right
            t = c.table.clone()
            t[t0, t1] = c.k.shape[0] if t0 else -1
            st, o2 = call(table=t)
            assert st == bad and torch.equal(o2[same], o[same])
        assert call(kv_len=[44, 2000, 21])[0] == bad and call(kv_len=[-1, 50, 21])[0] == bad
        for g in ([0, 2, 2], [0, 4, 3], [1, 2, 3], [0, -1, 3], [0, 2, 4]):
            assert call(groups=g)[0] == bad, g
        for p in ([41, 20], [-1, 20], [40, 2000]):
            assert call(prefix=p)[0] == bad, p
        assert call(max_own_len=9)[0] == bad and call(max_prefix_len=39)[0] == bad
        assert call(cu=[0, 4, 2, 3])[0] == bad and call(cu=[1, 1, 2, 3])[0] == bad


@TYPES
def test_shared_attention_is_paged_attention(dt):
    # every sequence a group without a prefix, and one prefix for all, against the call without groups
    r = Rand(61)
    hq, hk, dim, ps = 8, 2, 128, 16
    groups = [(200, [(1, 10 * i) for i in range(12)])]
    lens, kv, of, pre, bounds = shared_sizes(groups)
    c = SharedCache(r, [(pre[0], kv)], ps, hk, dim, dt)
    q = r.n(sum(lens), hq, dim, dt=dt)
    cut, kvt = ints(cu_of(lens)), ints(kv)
    want, wl = G().gdn_paged_attn(q, c.k, c.v, c.table, cut, kvt, lse=True)
    one = G().gdn_shared_attn(q, c.k, c.v, c.table, cut, kvt, ints(of), ints(pre), lse=True)
    alone = G().gdn_shared_attn(q, c.k, c.v, c.table, cut, kvt, ints(list(range(13))), ints([0] * 12), lse=True)
    whole = G().gdn_shared_attn(q, c.k, c.v, c.table, cut, kvt, ints(list(range(13))), ints(kv), lse=True)
    for o, l in (one, alone, whole):                             # each is within its own tolerance of the formula
        shared_check(c, q, o, l, lens, kv, dim ** -0.5, dt)
        assert (o.double() - want.double()).abs().max() <= 4 * R.u(dt) * c.vals[0].double().abs().max() + 1e-4
        assert (l - wl).abs().max() <= 1e-3


# ------------------------------------------------------------------ the next token
def settings(rows, T=None, k=None, p=None, m=None):
    def f(v, dt=F32):
        return None if v is None else torch.tensor(v if isinstance(v, list) else [v] * rows, dtype=dt, device="cuda")

    return dict(temperature=f(T), top_k=f(k, torch.int32), top_p=f(p), min_p=f(m))


def draw_check(x, u, s, skip_near=2.0 ** -34, most_near=None):
    """Tokens equal; logprob: the rounding to fp32, and the masses' 2^-36 (three of them)."""
    rows = x.shape[0]
    ws = new_ws(G().gdn_sample_workspace_bytes(G().make_sample_desc(x)))
    token, lp = G().gdn_sample(x, u, logprob=True, ws=ws, **s)
    assert G().gdn_device_status(ws) == 0 and token.dtype == torch.int32
    near = 0
    for i in range(rows):
        T, k, p, m = (d if s[n] is None else s[n][i].item() for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)))
        want, l, margin = PR.draw(x[i], u[i].item(), T, k, p, m)
        what = "row %d: T %r k %r p %r min-p %r u %r" % (i, T, k, p, m, u[i].item())
        if margin < skip_near:                                   # the documented border
            near += 1
            continue
        assert token[i].item() == want, what + ": got %d, want %d" % (token[i].item(), want)
        assert lp[i].item() == l or abs(lp[i].item() - l) <= R.U32 * abs(l) + 3 * 2.0 ** -36, what + ": %r %r" % (lp[i].item(), l)
    assert near <= (rows // 8 if most_near is None else most_near)
    return token, lp


@TYPES
@pytest.mark.parametrize("vocab,rows", [(1, 2), (2, 5), (63, 9), (2047, 4), (2049, 4), (8193, 3), (32000, 6), (70001, 4)])
def test_sample(dt, vocab, rows):
    r = Rand(vocab)
    x = r.n(rows, vocab, scale=3.0).to(dt)
    u = torch.rand(rows, generator=r.g).cuda()
    say("sample", dt, vocab, rows)
    draw_check(x, u, settings(rows))
    for T in (0.0, 0.05, 0.7, 2.0):
        draw_check(x, u, settings(rows, T=T))
        draw_check(x, u, settings(rows, T=T, k=min(40, vocab + 3), p=0.9, m=0.02))
    draw_check(x, u, settings(rows, k=1)), draw_check(x, u, settings(rows, k=vocab)), draw_check(x, u, settings(rows, k=vocab // 2 + 1))
    for p in (1e-7, 0.3, 0.999):
        draw_check(x, u, settings(rows, p=p))
    for m in (1.0, 0.5, 1e-6, 1e-30):
        draw_check(x, u, settings(rows, m=m))


@TYPES
def test_sample_settings_of_every_row(dt):
    r = Rand(7)
    rows, vocab = 64, 5003
    x = r.n(rows, vocab, scale=2.5).to(dt)
    g = random.Random(3)
    s = settings(rows, T=[g.choice([0.0, 0.3, 1.0, 1.7]) for _ in range(rows)], k=[g.choice([0, 1, 5, 400, 9000]) for _ in range(rows)],
                 p=[g.choice([1.0, 0.5, 0.95]) for _ in range(rows)], m=[g.choice([0.0, 0.1, 0.001]) for _ in range(rows)])
    u = torch.tensor([g.choice([0.0, 0.25, 1.0 - 2.0 ** -24, g.random()]) for _ in range(rows)], device="cuda")
    token, lp = draw_check(x, u, s)
    t2 = torch.full((rows,), 9, dtype=torch.int32, device="cuda")
    assert G().gdn_sample(x, u, token=t2, **s) is t2 and torch.equal(t2, token)


@TYPES
@pytest.mark.parametrize("offset,stride", [(0, 50), (1, 0), (3, 7), (5, 8), (7, 1)])
def test_sample_rows_that_start_anywhere(dt, offset, stride):
    r = Rand(offset)
    rows, vocab = 5, 4100
    wide = torch.full((rows, vocab + offset + stride), 50.0, dtype=dt, device="cuda")     # neighbours that would win
    x = wide[:, offset:offset + vocab]
    x.copy_(r.n(rows, vocab, scale=2.0))
    u = torch.rand(rows, generator=r.g).cuda()
    draw_check(x, u, settings(rows)), draw_check(x, u, settings(rows, T=0.0)), draw_check(x, u, settings(rows, k=30, p=0.8))


@TYPES
@pytest.mark.parametrize("vocab", [9000, 40000])
def test_sample_ties_and_flat_rows(dt, vocab):
    # bins of many tokens: all equal, two values, and differences far below a bin.  No row is left out for lying on a
    # border: equal weights are equal whole numbers, so that u M = j w is met exactly, as in the formula
    r = Rand(vocab)
    rows = 6
    u = torch.tensor([0.0, 0.25, 0.5, 0.9, 1.0 - 2.0 ** -24, 0.123], device="cuda")
    flat = torch.full((rows, vocab), -2.5, dtype=dt, device="cuda")
    two = torch.where(torch.rand(rows, vocab, generator=r.g).cuda() < 0.4, 1.0, 1.25).to(dt)
    close = (1.0 + torch.randint(0, 40, (rows, vocab), generator=r.g).cuda() * (2.0 ** -7 if dt is BF else 2.0 ** -23)).to(dt)
    spread = r.n(rows, vocab).to(dt)
    for x, Ts in ((flat, (1.0, 1e-6)), (two, (1.0, 0.01)), (close, (1.0, 1e-5)), (spread, (100.0, 1e30))):
        for T in Ts:
            draw_check(x, u, settings(rows, T=T), 0.0)
            draw_check(x, u, settings(rows, T=T, k=vocab // 2, p=0.7), 0.0)
            draw_check(x, u, settings(rows, T=T, k=vocab - 1, m=0.5), 0.0)
            draw_check(x, u, settings(rows, T=T, p=0.31, m=0.9), 0.0)
            draw_check(x, u, settings(rows, T=T, k=7), 0.0)


@TYPES
def test_sample_values_at_the_types_ends(dt):
    r = Rand(11)
    rows, vocab = 8, 3001
    low = torch.finfo(dt).min
    x = r.n(rows, vocab, scale=2.0).to(dt)
    x[0, 5:] = -math.inf                                         # five tokens left
    x[1, :3000] = -math.inf                                      # one, the last
    x[2, ::2] = low
    x[3] = low                                                   # all at the lowest value: ties
    x[4, 17], x[4, 2000] = math.inf, math.inf                    # the highest value, twice
    x[5, ::3] = math.nan
    x[6, 100], x[6, 7] = torch.finfo(dt).max, -0.0
    x[7] = 0.0
    x[7, ::2] = -0.0                                             # the two zeros are equal
    u = torch.tensor([0.9, 0.5, 0.3, 0.7, 0.6, 0.2, 0.999, 0.4], device="cuda")
    for T in (0.0, 1e-38, 0.01, 1.0, 50.0):
        for more in (dict(), dict(k=3), dict(p=0.5), dict(m=0.3)):
            draw_check(x, u, settings(rows, T=T, **more))
    none = torch.full((2, vocab), -math.inf, dtype=dt, device="cuda")
    none[1] = math.nan
    for T in (0.0, 1.0):
        ws = new_ws(1 << 20)
        token, lp = G().gdn_sample(none, u[:2], logprob=True, ws=ws, **settings(2, T=T, p=0.9))
        assert token.tolist() == [-1, -1] and lp.tolist() == [-math.inf] * 2 and G().gdn_device_status(ws) == 0


def test_sample_reports_bad_settings():
    r = Rand(12)
    x, u = r.n(3, 100), torch.tensor([0.1, 0.5, 0.9], device="cuda")
    want = G().gdn_sample(x, u)
    for name, values in (("temperature", (-1.0, math.nan, math.inf)), ("top_k", (-1,)), ("top_p", (0.0, -0.5, 1.5, math.nan)),
                         ("min_p", (-0.1, 1.1, math.nan)), ("u", (1.0, -0.1, math.nan))):
        for v in values:
            s = settings(3, T=1.0, k=0, p=1.0, m=0.0)
            uu = u.clone()
            (uu if name == "u" else s[name])[1] = v
            ws = new_ws(1 << 20)
            token, lp = G().gdn_sample(x, uu, logprob=True, ws=ws, **s)
            assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT, (name, v)
            assert token.tolist() == [want[0].item(), -1, want[2].item()] and lp[1] == -math.inf


# ------------------------------------------------------------------ together
@TYPES
def test_steps_of_a_server(dt):
    """Requests behind two prefixes through five steps: tables and positions, norm + rotation + append, attention, a
    projection to logits and the next token, which decides the next step's input, against the same
    steps with tables built on the host, attention without groups and the reference's draw."""
    g = G()
    r = Rand(88)
    hq, hk, dim, ps, vocab = 8, 2, 64, 16, 500
    pre, of = [48, 160], [0, 3, 7]
    n, steps = 7, 5
    prompt = [5, 1, 20, 3, 17, 1, 40]
    hit = [0, 0, 0, 1, 1, 1, 1]
    total_pages = 80
    kc, vc = (torch.full((total_pages, ps, hk, dim), math.nan, dtype=dt, device="cuda") for _ in range(2))
    order = r.perm(total_pages).tolist()
    pt = torch.full((2, 10), -1, dtype=torch.int32)
    for i, p in enumerate(pre):
        for j in range(p // ps):
            pt[i, j] = page = order.pop()
            kc[page], vc[page] = r.n(ps, hk, dim, dt=dt), r.n(ps, hk, dim, dt=dt)
    ang = torch.arange(300).double()[:, None] * 10000.0 ** (-torch.arange(0, dim, 2).double() / dim)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    embed = [r.n(vocab, h, dim, dt=dt) for h in (hq, hk, hk)]
    head = r.n(hq * dim, vocab, scale=0.3)
    tokens = [r.perm(vocab)[:x].tolist() for x in prompt]
    us = torch.rand(steps, n, generator=r.g).cuda()
    st = settings(n, T=[0.0, 0.5, 1.0, 1.0, 0.8, 1.2, 0.7], k=[0, 0, 20, 0, 7, 0, 1], p=[1.0, 0.9, 1.0, 0.8, 1.0, 1.0, 1.0])

    def run(shared):
        K, V = kc.clone(), vc.clone()
        table, free = torch.full((n, 20), -1, dtype=torch.int32, device="cuda"), ints(order)
        kv, at = ints([0] * n), ints([0])
        host = dict(table=table.tolist(), kv=[0] * n, at=0)
        new, ids, got = prompt, tokens, []
        for step in range(steps):
            T = sum(new)
            first = step == 0
            if shared:
                pr = dict(prefix_of=ints(hit), prefix_table=pt.cuda(), prefix_len=ints(pre)) if first else {}
                cu, kv, at, slots, pos = g.gdn_cache_extend(ints(new), kv, table, free, at, ps, T + 3, kv_out=kv, free_out=at, **pr)
                pos = pos[:T]
            else:
                t, c, k, a, _, p = PR.extend(new, host["kv"], host["table"], order, host["at"], ps, T, hit if first else None, pt.tolist(), pre)
                host = dict(table=t, kv=k, at=a)
                table, cu, kv, pos = ints(t), ints(c), ints(k), ints(p)
            flat = torch.tensor(sum(ids, []), device="cuda")
            q, k, v = (e[flat] for e in embed)
            qr = g.gdn_qk_norm_rope(q, k, v, cs, K, V, table, cu, kv, positions=pos)
            if shared:
                o = g.gdn_shared_attn(qr, K, V, table, cu, kv, ints(of), ints(pre))
            else:
                o = g.gdn_paged_attn(qr, K, V, table, cu, kv)
            logits = o[cu[1:].long() - 1].reshape(n, -1).float() @ head
            if shared:
                token = g.gdn_sample(logits, us[step], **st)
            else:
                token = ints([PR.draw(logits[i], us[step, i].item(), *(st[m][i].item() for m in ("temperature", "top_k", "top_p")))[0] for i in range(n)])
            got.append((token.tolist(), o, kv.tolist(), table.tolist() if step == steps - 1 else None))
            ids, new = [[t] for t in token.tolist()], [1] * n
        return got

    for step, (a, b) in enumerate(zip(run(True), run(False))):
        # both attentions are within the operators' tolerances of the formula: bf16 some roundings of 2^-8
        rel = float((a[1].double() - b[1].double()).norm() / b[1].double().norm())
        say("  step %d: attention with and without groups, relative %.2e" % (step, rel))
        assert rel <= (6 * 2 ** -8 if dt is BF else 1e-4)
        assert a[0] == b[0] and a[2] == b[2] and a[3] == b[3]


def test_captured_steps_replay():
    """All three in one graph, replayed between eager work, bit for bit."""
    g = G()
    r = Rand(91)
    hq, hk, dim, ps = 4, 2, 64, 16
    groups = [(100, [(1, 3), (1, 40)]), (33, [(1, 7)])]
    lens, kv, of, pre, bounds = shared_sizes(groups)
    c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], ps, hk, dim, BF)
    q = r.n(3, hq, dim, dt=BF)
    x, u = r.n(3, 20000, scale=3.0), torch.rand(3, generator=r.g).cuda()
    st = settings(3, T=0.8, k=50, p=0.95, m=0.01)
    ec = extend_case(92, 30, 16, 20, 2)
    T = sum(ec["new"])
    table0 = ints(ec["table"])
    new, kvi, free, at, table = ints(ec["new"]), ints(ec["kv"]), ints(ec["free"]), ints([ec["at"]]), table0.clone()
    big = extend_case(93, 700, 16, 20, 0)
    bnew, bkv, bfree, bat, btable = ints(big["new"]), ints(big["kv"]), ints(big["free"]), ints([big["at"]]), ints(big["table"])
    ofs = dict(prefix_of=ints(ec["hit"]), prefix_table=ints(ec["pt"]), prefix_len=ints(ec["pre"]))
    i32 = dict(dtype=torch.int32, device="cuda")
    bufs = dict(o=torch.empty_like(q), lse=torch.empty(3, hq, device="cuda"), token=torch.empty(3, **i32), lp=torch.empty(3, device="cuda"),
                cu=torch.empty(31, **i32), kvo=torch.empty(30, **i32), fo=torch.empty(1, **i32), slots=torch.empty(T, dtype=torch.int64, device="cuda"),
                pos=torch.empty(T, **i32), bcu=torch.empty(701, **i32), bkvo=torch.empty(700, **i32), bslots=torch.empty(8000, dtype=torch.int64, device="cuda"))
    wss = [new_ws(1 << 24) for _ in range(4)]
    cut, kvt, oft, pret = ints(cu_of(lens)), ints(kv), ints(of), ints(pre)

    def calls():
        g.gdn_cache_extend(new, kvi, table, free, at, ps, T, kv_out=bufs["kvo"], free_out=bufs["fo"], cu_seqlens=bufs["cu"], slots=bufs["slots"],
                           positions=bufs["pos"], ws=wss[0], **ofs)
        g.gdn_cache_extend(bnew, bkv, btable, bfree, bat, ps, 8000, kv_out=bufs["bkvo"], cu_seqlens=bufs["bcu"], slots=bufs["bslots"], positions=None, ws=wss[1])
        g.gdn_shared_attn(q, c.k, c.v, c.table, cut, kvt, oft, pret, o=bufs["o"], lse=bufs["lse"], ws=wss[2], **bounds)
        g.gdn_sample(x, u, token=bufs["token"], logprob=bufs["lp"], ws=wss[3], **st)

    calls()
    torch.cuda.synchronize()
    want, wt, wbt = {n: b.clone() for n, b in bufs.items()}, table.clone(), btable.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    a = torch.randn(256, 256, device="cuda")
    for rep in range(3):
        for b in bufs.values():
            b.fill_(-5)
        table.copy_(table0)
        (a @ a).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, b in bufs.items():
            assert torch.equal(b, want[name]), (rep, name)
        assert torch.equal(table, wt) and torch.equal(btable, wbt)
    assert all(g.gdn_device_status(ws) == 0 for ws in wss)


def test_two_streams_at_once():
    g = G()
    r = Rand(95)
    groups = [(300, [(1, 3), (1, 40), (1, 0)])]
    lens, kv, of, pre, bounds = shared_sizes(groups)
    c = SharedCache(r, [(300, kv)], 16, 2, 64, BF)
    q = [r.n(3, 8, 64, dt=BF) for _ in range(2)]
    x, u = [r.n(9, 30000, scale=3.0) for _ in range(2)], torch.rand(9, generator=r.g).cuda()
    args = (ints(cu_of(lens)), ints(kv), ints(of), ints(pre))
    wss = [[new_ws(1 << 24), new_ws(1 << 24)] for _ in range(2)]

    def calls(i, stream):
        return (g.gdn_shared_attn(q[i], c.k, c.v, c.table, *args, ws=wss[i][0], stream=stream, **bounds),
                g.gdn_sample(x[i], u, ws=wss[i][1], stream=stream, **settings(9, T=0.9, k=30)))

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[calls(i, streams[i]) for i in range(2)] for _ in range(5)]
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(p, w) for p, w in zip(a, b))
