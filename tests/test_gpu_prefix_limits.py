"""GPU: calls at the limits of what the operators around a prefix cache allow."""
import math

import pytest
import torch

import ops_reference as R
import prefix_reference as PR
from gpu_helpers import say
from test_gpu_ops import BF, F32, TYPES, Rand, cu_of, ints, new_ws  # noqa: F401
from test_gpu_prefix import SharedCache, extend_call, extend_case, draw_check, settings, shared_check

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


# ------------------------------------------------------------------ shared prefixes
@TYPES
@pytest.mark.parametrize("lens", [[1, 1, 1], [40, 1, 2]])
def test_shared_attention_reports_bad_input_without_own_keys(dt, lens):
    # the bounds leave no own keys, or no keys at all: no block but the join's looks at a sequence
    hq, hk, dim, pre = 4, 2, 64, [40, 30]
    kv = [40, 40, 30]
    c = SharedCache(Rand(3), [(40, kv[:2]), (30, kv[2:])], 16, hk, dim, dt)
    q = Rand(4).n(sum(lens), hq, dim, dt=dt)

    def status(kv_len, prefix=pre, groups=(0, 2, 3), max_kv_len=40, max_prefix_len=40):
        ws = new_ws(1 << 22)
        o, lse = G().gdn_shared_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv_len), ints(list(groups)), ints(prefix), lse=True, ws=ws,
                                     max_kv_len=max_kv_len, max_prefix_len=max_prefix_len, max_own_len=0)
        return G().gdn_device_status(ws), o, lse

    bad = G().GDN_ERR_DEVICE_INPUT
    st, o, lse = status(kv)
    assert st == 0
    shared_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)
    for i in range(3):
        for v in (-1, kv[i] + 1, 41, 1000):                      # negative, longer than its prefix, than max_kv_len
            assert status(kv[:i] + [v] + kv[i + 1:])[0] == bad, (i, v)
    for p in ([-1, 30], [41, 30], [40, 29]):
        assert status(kv, p)[0] == bad, p
    assert status([0, 0, 0], [0, 0], max_kv_len=0, max_prefix_len=0)[0] == 0
    for k, p in (([0, 0, 1], [0, 0]), ([-1, 0, 0], [0, 0]), ([0, 0, 0], [0, 1]), ([0, 0, 0], [-1, 0])):
        assert status(k, p, max_kv_len=0, max_prefix_len=0)[0] == bad, (k, p)


@TYPES
@pytest.mark.parametrize("hq,dim,lens,kv,pre,of", [
    (8, 64, [1, 1], [30, 35], [40], [0, 2]),                     # every kv_len below the prefix
    (8, 64, [3, 40, 1, 2], [30, 70, 5, 90], [100, 64], [0, 2, 4]),
    (4, 256, [1, 2, 1], [1, 500, 90], [600], [0, 3]),
    (2, 128, [1, 1, 1], [0, 0, 0], [64], [0, 3]),                # nothing is cached yet
])
def test_shared_attention_with_tight_bounds_below_the_prefix(dt, hq, dim, lens, kv, pre, of):
    r = Rand(dim + len(kv))
    c = SharedCache(r, [(p, kv[of[i]:of[i + 1]]) for i, p in enumerate(pre)], 16, 1, dim, dt)
    q = r.n(sum(lens), hq, dim, dt=dt)
    own = max(max(k - pre[i], 0) for i in range(len(pre)) for k in kv[of[i]:of[i + 1]])
    for bounds in (dict(max_kv_len=max(kv), max_prefix_len=max(pre), max_own_len=own), dict(max_kv_len=max(kv), max_prefix_len=max(pre)),
                   dict(max_kv_len=max(kv), max_prefix_len=1 << 20, max_own_len=1 << 20), dict(max_prefix_len=max(pre), max_own_len=own)):
        say("tight", dt, hq, dim, kv, pre, bounds)
        ws = new_ws(G().gdn_shared_workspace_bytes(G().make_shared_desc(q, c.k, c.table, len(kv), len(pre), **bounds)))
        o, lse = G().gdn_shared_attn(q, c.k, c.v, c.table, ints(cu_of(lens)), ints(kv), ints(of), ints(pre), lse=True, ws=ws, **bounds)
        assert G().gdn_device_status(ws) == 0, bounds
        shared_check(c, q, o, lse, lens, kv, dim ** -0.5, dt)


FINE = [  # h_kv, query heads of each, d, requests, groups: a token of each, whose prefix takes the form of 128 or 256 rows
    (2, 8, 64, 32, 2), (2, 8, 64, 64, 1), (1, 8, 128, 32, 4), (1, 8, 128, 64, 1), (1, 8, 256, 32, 2), (1, 8, 256, 64, 1)]


@pytest.mark.parametrize("hk,per,dim,n,n_groups", FINE)
def test_shared_attention_keeps_the_precision_of_few_rows(hk, per, dim, n, n_groups):
    # Two kinds of keys in turn, of probabilities 1 and 0.5016 before the division.  0.5016 is nearly half a bf16 step off
    # 0.5, and the values, 1 and -0.5, nearly cancel, so that rounding P to bf16 once would be off by as much as the output
    # itself, 1e-3.  Probabilities of 16 bits are off by 2^-16 relatively, 7e-6 of these outputs' sum of absolutes.
    ps, P, scale = 16, 700, 0.69003
    kc, vc = torch.zeros(9, ps, hk, dim, dtype=BF, device="cuda"), torch.full((9, ps, hk, dim), -0.5, dtype=BF, device="cuda")
    kc[:, 1::2, :, 0] = 1.0                                      # every page holds the same
    vc[:, 0::2] = 1.0
    vc[..., 1::2] *= -1.0
    q = torch.zeros(n, hk * per, dim, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    table = (torch.arange(n * 2000, dtype=torch.int32) * 7 % 9).view(n, 2000).cuda()
    kv = [P + 1 + i % 5 for i in range(n)]
    cu, of = cu_of([1] * n), [n // n_groups * g for g in range(n_groups + 1)]
    for pre in (P, 37):
        ws = new_ws(1 << 28)
        # the bound decides the form
        o = G().gdn_shared_attn(q, kc, vc, table, ints(cu), ints(kv), ints(of), ints([pre] * n_groups), scale=scale, ws=ws, max_prefix_len=31744,
                                max_own_len=700, max_kv_len=31744)
        assert G().gdn_device_status(ws) == 0
        whole = G().gdn_paged_attn(q, kc, vc, table, ints(cu), ints(kv), scale=scale, max_kv_len=max(kv))
        for i in range(5):
            keys, vals = (R.d(c[table[i, :45].long()].flatten(0, 1)[:kv[i]]) for c in (kc, vc))
            ref, oa, _, big = R.attend(R.d(q[i]), keys, vals, kv[i] - 1, scale)
            # as attn_tols, but for 16 bits of P where that counts 8
            off = 2 * (dim + 4) * R.U32 * big + (kv[i] + 8) * R.U32
            tol = R.u(BF) * ref.abs() + (off[:, None] + 2.0 ** -16) * (1 + 2 ** -6) * oa
            for j in range(i, n, 5):
                R.within(o[j], ref, tol, "request %d" % j)
                R.within(whole[j], ref, tol, "request %d, without groups" % j)


# ------------------------------------------------------------------ the next token
@TYPES
@pytest.mark.parametrize("width", [32768, 131072])
def test_sample_flat_rows_with_loose_ends(dt, width):
    # every token of the row is about the border, whole 16-byte pieces reach to its end, and elements lie in front of the
    # first one: the last turn of looking the row through lists 16 tokens a thread and the ends
    us = [0.0, 0.25, 0.51, 0.9, 1.0 - 2.0 ** -24]
    u = torch.tensor(us, device="cuda")
    for offset in (1, 2, 3):
        x = torch.zeros(5, width, dtype=dt, device="cuda")[:, offset:]
        vocab = width - offset
        say("flat", dt, width, offset)
        # equal weights: token j is the first with j + 1 > u n, n tokens staying
        for kw, n in ((dict(), vocab), (dict(k=vocab - 5), vocab - 5), (dict(k=vocab // 2), vocab // 2), (dict(T=100.0, p=0.5), -(-vocab // 2)), (dict(m=0.5), vocab)):
            token = G().gdn_sample(x, u, **settings(5, **kw))
            want = [int(v * n) for v in u.double().tolist()]
            assert token.tolist() == want, (dt, width, offset, kw)
    # a temperature at which all tokens are of one bin
    x = Rand(width).n(5, width, scale=2.0).to(dt)[:, 1:]
    for kw in (dict(), dict(k=width // 2, p=0.7)):
        draw_check(x, u, settings(5, T=1e30, **kw), 0.0)


@TYPES
def test_sample_flat_rows_of_odd_length(dt):
    # contiguous rows, of which each starts at another place in 16 bytes
    u = torch.linspace(0.0, 0.99, 9).cuda()
    for vocab in (32767, 32761, 49151):
        x = torch.zeros(9, vocab, dtype=dt, device="cuda")
        say("flat", dt, vocab)
        assert G().gdn_sample(x, u).tolist() == [int(v * vocab) for v in u.double().tolist()]


@TYPES
@pytest.mark.parametrize("vocab", [5, 1000, 2049, 40000])
def test_sample_at_the_highest_temperatures(dt, vocab):
    # 33 T passes the largest number: -inf, in the row and where its last chunk has no elements, is still no token
    rows = 6
    x = Rand(vocab).n(rows, vocab + 1, scale=2.0).to(dt)[:, 1:]
    top = torch.finfo(dt).max
    x[1, 1::2] = -math.inf
    x[2, 3:] = -math.inf
    x[3, 1:] = -top                                              # weights of 1 and, at T = 3.4e38, 1 / e
    x[3, 0] = 0.0
    x[4] = -top
    x[4, ::3] = -math.inf
    x[5, 0], x[5, 1] = top, -top
    u = torch.tensor([0.9, 0.6, 0.999, 0.3, 0.7, 0.45], device="cuda")
    # what counts as 0, weights under e^-32 of the largest, is less than vocab e^-32 of the mass (at T = 1e37 the lowest
    # numbers weigh e^-33.9 beside 0): a border is so much further off, in mass, and a logprob ln(1 + that) at most
    lost = vocab * math.exp(-32.0)
    for T in (1e25, 1.0e37, 1.04e37, 1e38, torch.finfo(F32).max):
        for kw in (dict(), dict(k=vocab - 1), dict(k=3), dict(p=0.6), dict(m=0.5), dict(m=0.2, p=0.9, k=vocab - 1)):
            s = settings(rows, T=T, **kw)
            token, lp = G().gdn_sample(x, u, logprob=True, **s)
            for i in range(rows):
                want, l, margin = PR.draw(x[i], u[i].item(), *(0 if s[n] is None and n == "top_k" else {"top_p": 1.0, "min_p": 0.0}[n] if s[n] is None
                                                              else s[n][i].item() for n in ("temperature", "top_k", "top_p", "min_p")))
                what = "T %r %r row %d: %d %r, want %d %r" % (T, kw, i, token[i].item(), lp[i].item(), want, l)
                # equal weights meet borders exactly; else what lies nearer than the documented accuracy is left out
                if 0.0 < margin < 2.0 ** -34 + lost:
                    continue
                assert token[i].item() == want, what
                assert abs(lp[i].item() - l) <= R.U32 * abs(l) + 3 * 2.0 ** -36 + lost, what


@TYPES
def test_sample_workspace_of_the_largest_batch(dt):
    r = Rand(49999)
    x, u = r.n(60, 49999, scale=2.0).to(dt), torch.rand(60, generator=r.g).cuda()
    st = settings(60, T=0.9, k=50, p=0.9)
    ws = new_ws(G().gdn_sample_workspace_bytes(G().make_sample_desc(x)))
    want = G().gdn_sample(x, u, **st)
    for rows in (60, 57, 20, 1):
        assert torch.equal(G().gdn_sample(x[:rows], u[:rows], ws=ws, **{n: v if v is None else v[:rows] for n, v in st.items()}), want[:rows])
    assert G().gdn_device_status(ws) == 0


def draw_of_classes(values, counts, u, T, k, p, m):
    """The draw from counts[c] tokens of each of the falling logits values[c] -> (class, place in it, how far u and p are from
    a border, in mass).  Sums of few products, exact to 2^-50 however many tokens there are."""
    w = [math.exp((v - values[0]) / T) for v in values]
    n, left = [], k or sum(counts)
    for c in counts:
        n.append(min(c, left))
        left -= n[-1]

    def border(target):
        front = 0.0
        for c, (a, b) in enumerate(zip(n, w)):
            if front + a * b > target:
                return c, (target - front) / b
            front = math.fsum(x * y for x, y in zip(n[:c + 1], w))
        return len(n) - 1, float(n[-1])

    margin = 1.0
    if p < 1.0:
        mass = math.fsum(a * b for a, b in zip(n, w))
        c, at = border(p * mass)
        margin = abs(at - round(at)) * w[c] / mass
        n = n[:c] + [math.ceil(at)]                              # the first so many that reach p of the mass
    n = [a if b >= m else 0 for a, b in zip(n, w)]
    mass = math.fsum(a * b for a, b in zip(n, w))
    c, at = border(u * mass)
    return c, math.floor(at), min(margin, abs(at - round(at)) * w[c] / mass), math.log(w[c] / mass)


@TYPES
def test_sample_accuracy_of_the_largest_vocabulary(dt):
    # the stated 2^-34, at 2^24 tokens: of few thousand different logits, whose masses are known exactly from their counts
    rows, vocab = 3, 1 << 24
    r = Rand(24)
    x = (r.n(rows, vocab + 3, scale=1.5).to(BF) + 0.0).to(dt)[:, 3:]
    x[1] = (x[1] * 0.25).to(BF).to(dt) + 0.0
    classes = [torch.unique(row.float(), return_counts=True) for row in x]
    classes = [(v.flip(0).tolist(), c.flip(0).tolist()) for v, c in classes]
    near = 0
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.8, 9000000, 0.7, 0.0), (1.3, 0, 0.999, 0.01), (1.0, 0, 1.0, 0.2)):
        for _ in range(3):
            u = torch.rand(rows, generator=r.g).cuda()
            s = settings(rows, T=T, k=k, p=p, m=m)
            token, lp = G().gdn_sample(x, u, logprob=True, **s)
            for i, (values, counts) in enumerate(classes):
                c, at, margin, l = draw_of_classes(values, counts, u[i].item(), *(s[a][i].item() for a in ("temperature", "top_k", "top_p", "min_p")))
                say("  T %g k %d p %g m %g row %d: place %d of %d, %.1e from a border" % (T, k, p, m, i, at, counts[c], margin))
                if margin < 2.0 ** -34:
                    near += 1
                    continue
                assert token[i].item() == (x[i].float() == values[c]).nonzero()[at].item(), (T, k, p, m, i)
                # the rounding to fp32, and the weight's and the mass's 1.13 2^-36 each
                assert abs(lp[i].item() - l) <= R.U32 * abs(l) + 3 * 2.0 ** -36
    assert near <= 3


# ------------------------------------------------------------------ block tables
@pytest.mark.parametrize("n,total", [(20, 0), (20, 5000), (1500, 0)])
def test_extend_with_an_empty_prefix_table(n, total):
    # no prefix is there: a request that names one is out of range, and -1 is none as ever
    c = extend_case(101, n, 16, 6)
    T = max(sum(c["new"]), total)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    for shape in ((0, 4), (0, 0)):
        for hit, where in ((-1, 0), (0, 0), (0, n - 1), (3, n // 2), (-2, 1)):
            of = [-1] * n
            of[where] = hit
            ws = new_ws(G().gdn_extend_workspace_bytes(n))
            out = extend_call(c, T, ws, prefix_of=ints(of), prefix_table=z.view(*shape), prefix_len=z)
            if hit == -1:
                assert G().gdn_device_status(ws) == 0
                want = PR.extend(c["new"], c["kv"], c["table"], c["free"], c["at"], 16, T)
                assert [x.tolist() for x in out] == [[w] if i == 3 else w for i, w in enumerate(want)]
            else:
                assert G().gdn_device_status(ws) == G().GDN_ERR_DEVICE_INPUT, (n, hit, where)
                table, cu, kv, at, slots, positions = out
                assert table.tolist() == c["table"] and cu.tolist() == [0] * (n + 1) and kv.tolist() == c["kv"] and at.tolist() == [c["at"]]
                assert (slots == -1).all() and (positions == -1).all()
