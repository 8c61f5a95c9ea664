"""GPU: every form that the operators around a prefix cache have, and the ends of their ranges.

The forms follow from the bounds of a call, so that loose bounds reach them with few keys."""
import math
import random

import pytest
import torch

import ops_reference as R
import prefix_reference as PR
from gpu_helpers import say
from test_gpu_ops import BF, F32, TYPES, Rand, attn_tols, cu_of, ints, new_ws
from test_gpu_prefix import SharedCache, draw_check, extend_call, extend_case, settings, shared_check

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


FORMS = [  # types, h_q, h_kv, d, groups, requests, new tokens of each, bounds of the prefix and of the own keys
    # few rows on both sides: 16 or 32 of them, 2, 4 or 8 waves
    ("bf", 1, 1, 64, 1, 1, 1, 64, 5000), ("both", 1, 1, 64, 1, 1, 1, 12000, 0), ("bf", 32, 1, 64, 1, 1, 1, 64, 40), ("bf", 8, 1, 64, 1, 1, 4, 300, 5000),
    ("bf", 8, 1, 64, 1, 1, 4, 12000, 0), ("both", 1, 1, 128, 2, 3, 1, 300, 5000), ("bf", 1, 1, 128, 1, 1, 1, 12000, 0),
    ("both", 2, 1, 256, 1, 2, 1, 64, 1), ("bf", 32, 1, 256, 1, 1, 1, 64, 1), ("bf", 32, 1, 256, 1, 1, 1, 300, 1), ("bf", 8, 1, 256, 1, 1, 4, 300, 0),
    ("f32", 1, 1, 64, 1, 1, 1, 300, 5000), ("f32", 2, 1, 128, 1, 2, 1, 64, 1), ("f32", 1, 1, 128, 1, 1, 1, 300, 1),
    # one side alone
    ("both", 6, 2, 64, 1, 3, 1, 0, 40), ("bf", 32, 1, 64, 1, 2, 1, 0, 5000), ("both", 8, 1, 256, 2, 3, 40, 0, 300), ("both", 6, 2, 128, 3, 5, 2, 300, 0),
    ("bf", 1, 1, 64, 1, 1, 40, 64, 0), ("bf", 1, 1, 256, 1, 200, 1, 64, 0), ("f32", 1, 1, 128, 1, 1, 40, 1000, 0),
    # many rows of the prefix, few of own keys
    ("bf", 32, 4, 64, 40, 100, 1, 1000, 1), ("bf", 6, 2, 64, 4, 64, 4, 12000, 4), ("bf", 16, 2, 64, 4, 64, 4, 12000, 300), ("bf", 32, 4, 128, 1, 200, 1, 12000, 4),
    ("bf", 32, 4, 256, 40, 200, 1, 300, 1), ("bf", 6, 2, 256, 4, 16, 4, 12000, 300), ("bf", 8, 2, 256, 1, 200, 1, 4000, 1000),
    ("f32", 32, 4, 64, 1, 64, 4, 64, 4), ("f32", 1, 1, 128, 1, 16, 40, 64, 300), ("f32", 1, 1, 128, 1, 16, 40, 1000, 300), ("f32", 1, 1, 256, 1, 1, 40, 1000, 40),
    # many on both
    ("bf", 1, 1, 64, 1, 1, 40, 64, 40), ("bf", 32, 1, 64, 1, 4, 4, 64, 4), ("bf", 8, 1, 128, 1, 1, 40, 64, 40), ("bf", 32, 1, 256, 1, 4, 4, 64, 4),
    ("f32", 1, 1, 64, 1, 1, 40, 1000, 1000), ("f32", 1, 1, 256, 1, 1, 40, 64, 1000),
]


@pytest.mark.parametrize("types,hq,hk,dim,n_groups,n,per,most_prefix,most_own", FORMS)
def test_shared_attention_forms(types, hq, hk, dim, n_groups, n, per, most_prefix, most_own):
    rnd = random.Random(n + most_prefix + most_own)
    ps = rnd.choice([1, 16, 20, 64])
    sizes = [len(range(i, n, n_groups)) for i in range(n_groups)]
    pre = [min(most_prefix, rnd.randrange(0, 70)) for _ in range(n_groups)]
    if most_prefix:
        pre[-1] = min(most_prefix, 64)
    # without own keys every position is in the prefix
    kv = [p + (rnd.randrange(per, min(most_own, 60) + 1) if most_own else 0) for p, s in zip(pre, sizes) for _ in range(s)]
    of, lens = cu_of(sizes), [per] * n
    for dt in {"bf": (BF,), "f32": (F32,), "both": (BF, F32)}[types]:
        r = Rand(n + hq + dim)
        c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], ps, hk, dim, dt)
        width = -(-(most_prefix + most_own) // ps)
        table = torch.full((n, width), -9, dtype=torch.int32, device="cuda")
        table[:, :min(width, c.table.shape[1])] = c.table[:, :width]
        q = r.n(n * per, hq, dim, dt=dt)
        bounds = dict(max_prefix_len=most_prefix, max_own_len=most_own)
        ws = new_ws(G().gdn_shared_workspace_bytes(G().make_shared_desc(q, c.k, table, n, n_groups, **bounds)))
        say("form", dt, hq, hk, dim, n_groups, n, per, most_prefix, most_own, "page", ps)
        o, lse = G().gdn_shared_attn(q, c.k, c.v, table, ints(cu_of(lens)), ints(kv), ints(of), ints(pre), lse=True, ws=ws, **bounds)
        assert G().gdn_device_status(ws) == 0
        shared_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)


@TYPES
def test_shared_attention_behind_32_bits(dt):
    """Pages behind 2^31 elements and 2^32 bytes of a cache."""
    r = Rand(70)
    ps, hk, dim, hq = 64, 2, 256, 4
    pages = 2 ** 31 // (ps * hk * dim) + 40
    cache = torch.empty(pages, ps, hk, dim, dtype=dt, device="cuda")
    pre, kv, lens = [70, 64], [75, 130, 66, 70], [1, 2, 1, 1]
    used = pages - 1 - r.perm(12)
    cache[used.cuda()] = r.n(12, ps, hk, dim, dt=dt)
    first = used.tolist()
    table = torch.full((4, 3), -1, dtype=torch.int32)
    table[0, :2], table[2, :2] = torch.tensor(first[:2]), torch.tensor(first[2:4])
    table[1, 1:], table[3, 1] = torch.tensor(first[4:6]), first[6]
    table[1, 0], table[3, 0] = first[0], first[2]
    # both hold the prefix's tail in their own pages: [64, 70) of group 0 are the first's
    cache[first[4], :6] = cache[first[1], :6]
    q = r.n(5, hq, dim, dt=dt)
    ws = new_ws(1 << 22)
    o, lse = G().gdn_shared_attn(q, cache, cache, table.cuda(), ints(cu_of(lens)), ints(kv), ints([0, 2, 4]), ints(pre), lse=True, ws=ws)
    assert G().gdn_device_status(ws) == 0
    keys = [cache[[p for p in row if p >= 0]].flatten(0, 1)[:n] for row, n in zip(table.tolist(), kv)]
    c = type("C", (), dict(keys=keys, vals=keys))
    shared_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)


# ------------------------------------------------------------------ the next token
@TYPES
def test_sample_of_a_large_vocabulary(dt):
    # parts of several units; bins of more tokens than the list takes, or than are looked at once, at every border
    vocab, rows = 600001, 6
    r = Rand(71)
    x = r.n(rows, vocab, scale=2.0).to(dt)
    x[4] = -1.0                                                  # ties over the whole row
    u = torch.tensor([0.99, 0.4, 0.7, 0.25, 0.6, 1.0 - 2.0 ** -24], device="cuda")
    s = settings(rows, T=[1.0, 30.0, 1.0, 3.0, 1.0, 0.3], k=[0, 0, 200000, 400000, 599999, 0], p=[1.0, 1.0, 0.93, 0.5, 0.75, 1.0],
                 m=[0.0, 0.0, 1e-4, 0.2, 0.0, 0.0])
    say("sample", dt, rows, vocab)
    # the last row's u leaves 2^-24 of the mass, which some 10^5 tokens share: each brings less than 2^-34 of the mass, so that
    # the border is that near by arithmetic
    draw_check(x, u, s, most_near=1)


@TYPES
@pytest.mark.parametrize("offset", [0, 3])
def test_sample_of_many_rows(dt, offset):
    # chunks of 8192 elements, whose last is short
    rows, vocab = 256, 8200
    r = Rand(72)
    x = r.n(rows, vocab + offset, scale=2.0).to(dt)[:, offset:]
    x[5, 8190:] = 9.0
    x[6, :8195] = -math.inf
    g = random.Random(4)
    s = settings(rows, T=[g.choice([0.0, 0.6, 1.0, 9.0]) for _ in range(rows)], k=[g.choice([0, 20, 6000]) for _ in range(rows)],
                 p=[g.choice([1.0, 0.4, 0.99]) for _ in range(rows)], m=[g.choice([0.0, 0.05]) for _ in range(rows)])
    say("sample", dt, rows, vocab, offset)
    draw_check(x, torch.rand(rows, generator=r.g).cuda(), s)


@TYPES
@pytest.mark.parametrize("sign", [1, -1])
def test_sample_borders_far_apart(dt, sign):
    # the filters' borders and the token in bins that do not touch, on either side of zero and on both
    rows, vocab = 8, 30000
    r = Rand(73)
    x = (sign * torch.rand(rows, vocab, generator=r.g).cuda() * 8 - (0 if sign > 0 else -2.0)).to(dt)
    u = torch.tensor([0.0, 1e-4, 0.01, 0.2, 0.5, 0.9, 0.999, 0.3], device="cuda")
    for kw in (dict(k=20000), dict(k=25000, p=0.99), dict(p=0.9), dict(m=0.01), dict(k=29000, p=0.995, m=0.002)):
        for T in (1.0, 2.5):
            draw_check(x, u, settings(rows, T=T, **kw))


@TYPES
def test_sample_bins_of_what_min_p_drops(dt):
    # min-p's border, and top-k's, in a bin whose tokens are all behind it.  They are counted, for their chunk's largest
    # logit is lower than the row's; the token's own bin holds too many for one look at both
    rows, vocab = 4, 5000
    r = Rand(76)
    x = torch.full((rows, vocab), -9.0)
    x[:, 3] = 0.0
    x[:, 2500:3100] = -0.5 + (torch.randint(0, 12, (rows, 600), generator=r.g) - 6) * 2.0 ** -8
    x[:, 4000:4010] = -1.03125
    u = torch.tensor([0.1, 0.5, 0.9, 0.999], device="cuda")
    for k in (0, 603, 611):
        for T, m in ((1.0, math.exp(-1.0)), (2.0, math.exp(-0.5))):
            draw_check(x.to(dt).cuda(), u, settings(rows, T=T, m=m, k=k))


@TYPES
def test_sample_few_tokens_of_which_min_p_drops_some(dt):
    # as above, with few tokens: all borders are looked at together, and a bin between the token's and theirs is not
    rows, vocab = 5, 5000
    x = torch.full((rows, vocab), -9.0)
    x[:, 3] = 0.0
    x[:, 2500:2505] = -0.5
    x[:, 3000:3004] = -0.75
    x[:, 4000:4010] = -1.03125
    u = torch.tensor([0.1, 0.3, 0.5, 0.9, 0.999], device="cuda")
    for k in (0, 1, 5, 8, 10, 12, 19):
        for T, m in ((1.0, math.exp(-1.0)), (2.0, math.exp(-0.5)), (1.0, 0.999), (1.0, math.exp(-0.52))):
            draw_check(x.to(dt).cuda(), u, settings(rows, T=T, m=m, k=k))


@TYPES
def test_sample_logprob_of_the_only_token_is_zero(dt):
    r = Rand(78)
    for vocab in (5, 3000, 70000):
        x = r.n(12, vocab, scale=3.0).to(dt)
        x[:, 2] = 40.0 + 0.25 * torch.arange(12).cuda()          # anywhere in a bin
        x[6:, 4] = 0.5 * x[6:, 2]                                # one more, of little weight
        u = torch.rand(12, generator=r.g).cuda()
        for kw in (dict(k=1), dict(p=1e-6), dict(m=1.0), dict(m=0.9, T=0.7), dict(k=1, p=0.5, m=0.1, T=3.0), dict(T=0.0), dict(T=1e-12)):
            token, lp = G().gdn_sample(x, u, logprob=True, **settings(12, **kw))
            assert (token == 2).all() and (lp == 0).all(), (vocab, kw, lp.tolist())


@TYPES
def test_sample_nan_beside_infinity(dt):
    # NaN is no token, also where the row's largest logit is +inf
    r = Rand(77)
    x = r.n(4, 3000).to(dt)
    x[0, 5], x[0, 2500] = math.nan, math.inf
    x[1, 100], x[1, 99] = math.inf, math.nan
    x[2, :] = math.nan
    x[2, 2999] = math.inf
    x[3, 7], x[3, 8] = math.nan, torch.finfo(dt).max
    for T in (0.0, 1e-3, 1.0):
        draw_check(x, torch.tensor([0.1, 0.4, 0.6, 0.9], device="cuda"), settings(4, T=T)), draw_check(x, torch.rand(4).cuda(), settings(4, T=T, k=4, p=0.9))


@TYPES
def test_sample_of_the_largest_vocabulary(dt):
    # 2^24 tokens, rows that start inside 16 bytes: every part of a row's bookkeeping at its end.  The order and the sums are
    # torch's in 64 bits; what a border of 2^-34 of the mass or nearer would decide is left out
    vocab = 1 << 24
    r = Rand(79)
    wide = r.n(3, vocab + 3, scale=1.5).to(dt)
    wide[1] = torch.rand(vocab + 3, generator=r.g).cuda().to(dt)
    x = wide[:, 3:]
    x[2, :] = -30.0
    x[2, vocab - 1], x[2, 5] = 1.0, -3.0
    u = torch.tensor([0.37, 0.81, 1.0 - 2.0 ** -20], device="cuda")
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (1.0, 9000000, 0.7, 0.0), (0.8, 0, 0.999, 0.01), (0.0, 0, 1.0, 0.0)):
        token, lp = G().gdn_sample(x, u, logprob=True, **settings(3, T=T, k=k, p=p, m=m))
        for i in range(3):
            if T == 0.0:
                assert token[i].item() == int(x[i].float().argmax()) if i == 2 else x[i, token[i]] == x[i].max()
                continue
            v, order = torch.sort(x[i].double(), descending=True, stable=True)
            w = ((v - v[0]) / T).exp().cpu()
            c = w.cumsum(0)
            n = min(k or vocab, vocab)
            if p < 1.0:
                n = int((c[:n] < c[n - 1] * settings(1, p=p)["top_p"].double().item()).sum()) + 1
            if m > 0.0:
                n = min(n, int((w >= settings(1, m=m)["min_p"].double().item()).sum()))
            want = u[i].double().item() * c[n - 1].item()
            at = int((c[:n] <= want).sum())
            near = min(abs(c[j].item() - want) for j in (at - 1, at) if j >= 0) / c[n - 1].item()
            say("  T %g k %d p %g m %g row %d: token %d of the order, %.1e from a border" % (T, k, p, m, i, at, near))
            # the sums here carry 2^24 roundings of 2^-53 and bins of so many tokens theirs, and p's border moves u's
            if near > 2.0 ** -26:
                assert token[i].item() == order[at].item()
            assert abs(lp[i].item() - math.log(w[at].item() / c[n - 1].item())) <= R.U32 * 20 + 2.0 ** -20


@TYPES
def test_sample_rows_behind_32_bits(dt):
    rows, vocab, stride = 3, 5000, 2 ** 30 + 8
    r = Rand(74)
    wide = torch.empty(2 * stride + vocab, dtype=dt, device="cuda")
    x = wide.as_strided((rows, vocab), (stride, 1))
    x.copy_(r.n(rows, vocab, scale=2.0))
    draw_check(x, torch.tensor([0.3, 0.6, 0.9], device="cuda"), settings(rows, T=0.8, k=900, p=0.9))


def test_one_workspace_for_calls_of_every_size():
    g = G()
    r = Rand(75)
    ws = new_ws(1 << 24)
    for rows, vocab in ((60, 50000), (1, 7), (300, 9000), (3, 70000), (1, 1), (60, 50000)):
        x, u = r.n(rows, vocab, scale=2.0), torch.rand(rows, generator=r.g).cuda()
        st = settings(rows, T=0.9, k=50, p=0.9)
        assert torch.equal(g.gdn_sample(x, u, ws=ws, **st), g.gdn_sample(x, u, **st)), (rows, vocab)
    assert g.gdn_device_status(ws) == 0


# ------------------------------------------------------------------ block tables
@pytest.mark.parametrize("n,empty", [(900, 0.97), (2500, 0.97), (2500, 1.0), (70000, 0.999)])
def test_extend_of_mostly_empty_steps(n, empty):
    c = extend_case(81, n, 16, 90, 3, empty=empty)
    T = sum(c["new"])
    ws = new_ws(G().gdn_extend_workspace_bytes(n))
    say("extend", n, empty, T)
    table, cu, kv, at, slots, positions = extend_call(c, T + 3, ws)
    want = PR.extend(c["new"], c["kv"], c["table"], c["free"], c["at"], 16, T + 3, c["hit"], c["pt"], c["pre"])
    assert G().gdn_device_status(ws) == 0
    for name, got, w in zip(("table", "cu", "kv", "at", "slots", "positions"), (table, cu, kv, at, slots, positions), want):
        assert got.tolist() == ([w] if name == "at" else w), name


@pytest.mark.parametrize("n", [5, 2000])
def test_extend_slots_behind_32_bits(n):
    c = extend_case(82, n, 128, 200, 0)
    c["free"] = [2 ** 31 - 1 - i for i in range(len(c["free"]))]
    T = sum(c["new"])
    out = extend_call(c, T)
    want = PR.extend(c["new"], c["kv"], c["table"], c["free"], c["at"], 128, T)
    assert out[4].tolist() == want[4] and max(want[4]) > 2 ** 37 and out[0].tolist() == want[0]


def test_extend_on_the_largest_positions():
    # kv_len up to the table's whole pages, one request
    ps, width = 1 << 20, 2000
    kv, new = ps * width - 3, 3
    table = torch.arange(width, dtype=torch.int32, device="cuda")[None].clone()
    cu, kv2, at, slots, positions = G().gdn_cache_extend(ints([new]), ints([kv]), table, ints([7]), ints([0]), ps, 3)
    assert kv2.tolist() == [ps * width] and at.tolist() == [0] and cu.tolist() == [0, 3]
    assert positions.tolist() == [kv, kv + 1, kv + 2] and slots.tolist() == [kv, kv + 1, kv + 2]
