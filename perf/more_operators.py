"""Operators around a prefix cache's steps: their workloads, plain forms and exact values.

A server that keeps prefixes runs three more things beside the suffix and decode operators.  The
step's bookkeeping (``extend``): lengths, block tables, packed offsets, positions and slots of the
new tokens, from the requests' new lengths, the prefixes that were hit and the free pages.  The
attention of a batch whose requests share prefixes (``attn``): a prefix's keys and values are the
same for all of a group's rows.  And the draw of the next token from the logits (``sample``):
temperature, top-k, top-p and min-p with given random numbers.
A case names its operator (``op``) and its sizes.  ``run`` computes it with elementary torch
operations, or with this package's calls where ``own`` is true; ``exact`` computes it in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the next token of two requests behind one short hit: the smallest attention
        dict(name="shared_two_requests", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=16, groups=1, n_seqs=2, tokens=2, spread=1, prefix=1024, own=60),
        # the next token of 64 requests behind one 31744-token prefix, up to 1K of their own
        dict(name="shared_next_token", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=64, groups=1, n_seqs=64, tokens=64, spread=2, prefix=31744, own=1024),
        # the next token of 96 requests behind 7 prefixes of different lengths, 8 cache heads
        dict(name="shared_groups", op="attn", dtype="bf16", h_q=32, h_kv=8, d=128, page=16, groups=7, n_seqs=96, tokens=96, spread=3, prefix=8192, own=1500),
        # suffixes of different lengths behind one 16K hit: prompts
        dict(name="shared_suffixes", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=64, groups=1, n_seqs=12, tokens=1501, spread=4, prefix=16384, own=0),
        # a few tokens of every request behind prefixes that end inside a page, fp32
        dict(name="shared_packed_f32", op="attn", dtype="f32", h_q=16, h_kv=4, d=64, page=24, groups=3, n_seqs=19, tokens=101, spread=5, prefix=4000, own=700),
        # the next token of one request, every filter on: the smallest draw
        dict(name="sample_one", op="sample", dtype="bf16", rows=1, vocab=32768, filters="all", masked=False),
        # 64 requests, each with settings of its own, over the fp32 logits of a large vocabulary
        dict(name="sample_batch", op="sample", dtype="f32", rows=64, vocab=131072, filters="mixed", masked=False),
        # 256 requests with settings of their own
        dict(name="sample_large", op="sample", dtype="bf16", rows=256, vocab=131072, filters="mixed", masked=False),
        # temperature alone, an odd vocabulary whose rows start anywhere, some of them masked by a grammar
        dict(name="sample_unfiltered", op="sample", dtype="bf16", rows=48, vocab=49999, filters="none", masked=True),
        # one more token of 64 running requests: the smallest step
        dict(name="extend_next_token", op="extend", n_seqs=64, tokens=64, page=16, spread=1, prefix=0, prefixes=0, context=8192),
        # a large batch of continuing requests and of new ones behind 5 prefixes, prompts in pieces
        dict(name="extend_prompts", op="extend", n_seqs=700, tokens=65536, page=16, spread=2, prefix=16384, prefixes=5, context=20000),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn", "attn", "attn", "sample", "sample", "extend"])
    if op == "sample":
        c = dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=log(1, 256), vocab=log(1000, 131072),
                 filters=rng.choice(["none", "all", "mixed", "mixed"]), masked=rng.random() < 0.3)
        while c["rows"] * c["vocab"] * _BYTES[c["dtype"]] > 256 * 131072 * 2:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    if op == "extend":
        n = log(1, 2000)
        c = dict(op=op, n_seqs=n, tokens=n if rng.random() < 0.4 else n + log(1, 60000), page=rng.choice([1, 16, 24, 32, 64, 128]),
                 spread=rng.randrange(1, 1000), prefixes=rng.choice([0, 1, 3, 8]), context=log(1, 20000))
        c["prefix"] = log(1, 16384) if c["prefixes"] else 0
        while n * (c["context"] + c["prefix"]) > 24000000 * min(16, c["page"]) // 16:
            c["context"], c["prefix"] = c["context"] // 2, c["prefix"] // 2
        return c
    dt = rng.choice(["bf16", "bf16", "f32"])
    half = 2 if dt == "f32" else 1
    kv, d, n = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), log(1, 96)
    c = dict(op=op, dtype=dt, h_q=kv * rng.choice([1, 2, 3, 4, 8]), h_kv=kv, d=d, page=rng.choice([1, 16, 24, 32, 64, 128, 256]),
             groups=rng.choice([1, 1, 2, 5, 9]), n_seqs=n, tokens=rng.choice([n, n, n + log(1, 1400)]), spread=rng.randrange(1, 1000),
             prefix=log(16, 32768 // half), own=log(1, 2000))
    # no dearer than the next token of 64 requests behind one prefix, or the suffixes
    while c["tokens"] * (c["prefix"] + c["own"]) * c["h_q"] * d * half * half > 1501 * 16384 * 16 * 256 \
            or (c["groups"] * c["prefix"] + n * c["own"]) * kv * d * half > 64 * 1024 * 1024:
        c["prefix"] = max(1, c["prefix"] // 2)
        c["own"] = max(1, c["own"] * 3 // 4)
        c["tokens"] = max(n, c["tokens"] * 3 // 4)
    return c


# ------------------------------------------------------------------ lengths
def _shares(total, n, seed):
    """`total` in n uneven parts, each at least one where that is possible."""
    if total == n:
        return [1] * n
    r = random.Random(seed * 7919 + n)
    w = [r.random() ** 2 for _ in range(n)]
    s = sum(w) or 1.0
    got = [1 + int((total - n) * x / s) for x in w]
    got[r.randrange(n)] += total - sum(got)
    return got


def _cu(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


def _attn_sizes(case):
    """(new tokens of each request, requests in front of each group, each group's prefix, each request's own cached tokens)."""
    n, g = case["n_seqs"], min(case["groups"], case["n_seqs"])
    r = random.Random(case["spread"] * 104729 + n)
    lens = _shares(case["tokens"], n, case["spread"])
    of = _cu(_shares(n, g, case["spread"] + 1))
    if g == 1:
        prefix = [case["prefix"]]
    else:  # the last group's requests share nothing
        prefix = [r.randrange(case["prefix"] // 16, case["prefix"] + 1) for _ in range(g - 1)] + [0]
    if case["spread"] % 2 == 0 or case["page"] == 1:  # hits of whole pages
        prefix = [x // case["page"] * case["page"] for x in prefix]
    return lens, of, prefix, [r.randrange(0, case["own"] + 1) for _ in range(n)]


def _extend_sizes(case):
    """(new tokens, tokens cached before, prefix hit or -1, of each request; each prefix's tokens)."""
    n, ps = case["n_seqs"], case["page"]
    r = random.Random(case["spread"] * 15485863 + n)
    lens = _shares(case["tokens"], n, case["spread"])
    pre = [r.randrange(0, case["prefix"] + 1) // ps * ps for _ in range(case["prefixes"])]
    hit = [r.randrange(len(pre)) if pre and r.random() < 0.5 else -1 for _ in range(n)]
    old = [0 if h >= 0 else r.randrange(0, case["context"] + 1) for h in hit]
    return lens, old, hit, pre


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = {"case": dict(case)}
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = normal(rows, vocab) * 2.2
        likely = torch.randint(0, vocab, (rows, 12), generator=g, device=DEV)  # what the context calls for
        x.scatter_add_(1, likely, uniform(rows, 12, lo=3.0, hi=11.0))
        if case["masked"]:  # a grammar leaves a few tokens to a part of the rows
            some = (uniform(rows, 1) < 0.5) & (uniform(rows, vocab) < 0.99)
            some[:, 0] = False
            x.masked_fill_(some, -math.inf)
        s["logits"], s["u"] = x.to(_DT[case["dtype"]]), torch.rand(rows, generator=g, device=DEV)
        s["temperature"] = uniform(rows, lo=0.5, hi=1.3)
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if case["filters"] != "none":
            def maybe(v, off):
                return torch.where(uniform(rows) < 0.4, off, v) if case["filters"] == "mixed" else v

            zero, one = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
            s["top_k"] = maybe(torch.exp(uniform(rows, lo=0.0, hi=math.log(min(1000, vocab)))).floor(), zero).to(torch.int32)
            s["top_p"], s["min_p"] = maybe(uniform(rows, lo=0.6, hi=0.99), one), maybe(uniform(rows, lo=0.0, hi=0.1), zero)
        if case["filters"] == "mixed":
            s["temperature"] = torch.where(uniform(rows) < 0.1, torch.zeros(rows, device=DEV), s["temperature"])
        if own:
            import gated_deltanet_state_gdn_amd as gdn
            s["ws"] = torch.zeros(gdn.gdn_sample_workspace_bytes(gdn.make_sample_desc(s["logits"])), dtype=torch.uint8, device=DEV)
        return s
    ps = case["page"]
    if case["op"] == "extend":
        lens, old, hit, pre = _extend_sizes(case)
        base = [pre[h] if h >= 0 else o for h, o in zip(hit, old)]
        have = [-(-o // ps) for o in old]
        need = [-(-(b + x) // ps) - -(-b // ps) for b, x in zip(base, lens)]
        most = max(-(-(b + x) // ps) for b, x in zip(base, lens)) + 3
        pages = torch.randperm(sum(have) + sum(need) + sum(x // ps for x in pre) + 100, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
        s["table"][torch.arange(most, device=DEV)[None] < ints(have)[:, None]] = pages[:sum(have)]
        s["prefix_table"] = s["prefix_len"] = s["prefix_of"] = None
        at = sum(have)
        if pre:
            s["prefix_table"] = torch.full((len(pre), max(x // ps for x in pre) + 1), -1, dtype=torch.int32, device=DEV)
            for i, x in enumerate(pre):
                s["prefix_table"][i, :x // ps] = pages[at:at + x // ps]
                at += x // ps
            s["prefix_len"], s["prefix_of"] = ints(pre), ints(hit)
        s["free"] = torch.cat([ints([0] * 7), pages[at:]])  # seven of the list are taken already
        s.update(new=ints(lens), kv=ints(old), at=ints([7]))
        if own:
            import gated_deltanet_state_gdn_amd as gdn
            s["ws"] = torch.zeros(gdn.gdn_extend_workspace_bytes(len(lens)), dtype=torch.uint8, device=DEV)
        return s
    lens, of, prefix, own_len = _attn_sizes(case)
    n, hk, d, dt = len(lens), case["h_kv"], case["d"], _DT[case["dtype"]]
    group = [i for i in range(len(prefix)) for _ in range(of[i], of[i + 1])]
    total = [prefix[group[i]] + own_len[i] + lens[i] for i in range(n)]
    # a prefix's whole pages are the same for its group; where it ends inside a page, each request has a copy of that
    whole = [x // ps for x in prefix]
    mine = [-(-total[i] // ps) - whole[group[i]] for i in range(n)]
    pages = sum(whole) + sum(mine) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((n, max(-(-x // ps) for x in total)), -1, dtype=torch.int32, device=DEV)
    s["kc"], s["vc"] = normal(pages, ps, hk, d, dtype=dt), normal(pages, ps, hk, d, dtype=dt)
    at = sum(whole)
    for i in range(n):
        j = group[i]
        front = sum(whole[:j])
        s["table"][i, :whole[j]] = order[front:front + whole[j]]
        s["table"][i, whole[j]:whole[j] + mine[i]] = order[at:at + mine[i]]
        at += mine[i]
        left = prefix[j] % ps
        if left and i > of[j]:
            first, here = s["table"][of[j], whole[j]].long(), s["table"][i, whole[j]].long()
            for c in (s["kc"], s["vc"]):
                c[here, :left] = c[first, :left]
    s["q"] = normal(case["tokens"], case["h_q"], d, dtype=dt)
    s.update(cu=ints(_cu(lens)), kv_len=ints(total), groups=ints(of), prefix_len=ints(prefix))
    s["bounds"] = dict(max_kv_len=max(total), max_prefix_len=max(prefix), max_own_len=max(total[i] - prefix[group[i]] for i in range(n)))
    if own:
        import gated_deltanet_state_gdn_amd as gdn
        desc = gdn.make_shared_desc(s["q"], s["kc"], s["table"], n, len(prefix), **s["bounds"])
        s["ws"] = torch.zeros(gdn.gdn_shared_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
    return s


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * _BYTES[case["dtype"]] + case["rows"] * 28, "flops": 4 * n}
    if case["op"] == "extend":
        lens, old, hit, pre = _extend_sizes(case)
        ps = case["page"]
        entries = sum(-(-((pre[h] if h >= 0 else o) + x) // ps) - (0 if h >= 0 else -(-o // ps)) for x, o, h in zip(lens, old, hit))
        return {"bytes": 20 * len(lens) + 8 * entries + 12 * sum(lens), "flops": 4 * sum(lens)}
    lens, of, prefix, own_len = _attn_sizes(case)
    t, hq, hk, d, e = case["tokens"], case["h_q"], case["h_kv"], case["d"], _BYTES[case["dtype"]]
    group = [i for i in range(len(prefix)) for _ in range(of[i], of[i + 1])]
    keys = sum(prefix) + sum(a + b for a, b in zip(lens, own_len))
    pairs = sum(x * (prefix[group[i]] + own_len[i]) + x * (x + 1) // 2 for i, x in enumerate(lens))
    return {"bytes": 2 * keys * hk * d * e + 2 * t * hq * d * e + t * hq * 4, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_attn(s):
    import gated_deltanet_state_gdn_amd as gdn
    o, lse = gdn.gdn_shared_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_len"], s["groups"], s["prefix_len"], lse=True, ws=s["ws"], **s["bounds"])
    return {"o": o, "lse": lse}


def _own_sample(s):
    import gated_deltanet_state_gdn_amd as gdn
    token, logprob = gdn.gdn_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                    logprob=True, ws=s["ws"])
    return {"token": token, "logprob": logprob}


def _own_extend(s):
    import gated_deltanet_state_gdn_amd as gdn
    cu, kv, at, slots, positions = gdn.gdn_cache_extend(s["new"], s["kv"], s["table"], s["free"], s["at"], s["case"]["page"], s["case"]["tokens"] + 8,
                                                        prefix_of=s["prefix_of"], prefix_table=s["prefix_table"], prefix_len=s["prefix_len"], ws=s["ws"])
    return {"table": s["table"], "cu": cu, "kv": kv, "at": at, "slots": slots, "positions": positions}


_own = {"attn": _own_attn, "sample": _own_sample, "extend": _own_extend}


def _plain_attn(s):
    lens, of, prefix, _ = _attn_sizes(s["case"])
    q, kc, vc, cu, kv = s["q"], s["kc"], s["vc"], s["cu"].long(), s["kv_len"].long()
    t, hq, d = q.shape
    ps, hk = kc.shape[1:3]
    rep = hq // hk
    at = _cu(lens)
    outs, ends = [], []
    for j, p in enumerate(prefix):
        a, b = of[j], of[j + 1]
        rows = q[at[a]:at[b]].float() * d ** -0.5
        n, most = b - a, max(lens[a:b])
        # the prefix, once for the group: [hk, rows, p]
        table = torch.clamp(s["table"][a:b], min=0).long()
        keys = kc[table[0]].view(-1, hk, d)[:p].float().permute(1, 2, 0)
        vals = vc[table[0]].view(-1, hk, d)[:p].float().transpose(0, 1)
        m = rows.shape[0]
        grouped = rows.view(m, hk, rep, d).transpose(0, 1).reshape(hk, m * rep, d)
        score = torch.matmul(grouped, keys)
        # each request's own keys: [n, hk, most rows, longest]
        longest = max(s["bounds"]["max_own_len"], 1)
        spot = p + torch.arange(longest, device=DEV)
        page = table[:, torch.clamp(spot // ps, max=table.shape[1] - 1)]
        ok = kc[page, spot % ps].float().permute(0, 2, 3, 1)
        ov = vc[page, spot % ps].float().transpose(1, 2)
        new = cu[a:b, None] + torch.arange(most, device=DEV)
        mine = (q[torch.clamp(new, max=t - 1)].float() * d ** -0.5).view(n, most, hk, rep, d).permute(0, 2, 1, 3, 4).reshape(n, hk, most * rep, d)
        pos = (kv[a:b] - cu[a + 1:b + 1])[:, None] + new
        seen = (spot <= pos[..., None]).repeat_interleave(rep, 1)[:, None]
        own_score = torch.matmul(mine, ok).masked_fill_(~seen, -math.inf)
        seq = torch.searchsorted(cu[a + 1:b + 1].contiguous(), torch.arange(at[a], at[b], device=DEV), right=True)
        back = seq * most + torch.arange(at[a], at[b], device=DEV) - cu[a:b][seq]

        def packed(v):  # [n, hk, most rep, x] -> [hk, m rep, x]
            x = v.shape[-1]
            return v.view(n, hk, most, rep, x).permute(1, 0, 2, 3, 4).reshape(hk, n * most, rep, x)[:, back].reshape(hk, m * rep, x)

        top = packed(own_score.amax(-1, keepdim=True))
        if p:
            top = torch.maximum(top, score.amax(-1, keepdim=True))
        wide = torch.full((n * most, hk, rep, 1), 0.0, device=DEV)
        wide[back] = top.view(hk, m, rep, 1).transpose(0, 1)
        own_score = torch.exp(own_score.sub_(wide.view(n, most, hk, rep, 1).permute(0, 2, 1, 3, 4).reshape(n, hk, most * rep, 1)))
        o, total = packed(torch.matmul(own_score, ov)), packed(own_score.sum(-1, keepdim=True))
        if p:
            score = torch.exp(score.sub_(top))
            o, total = o + torch.matmul(score, vals), total + score.sum(-1, keepdim=True)
        outs.append((o / total).view(hk, m, rep, d).transpose(0, 1).reshape(m, hq, d))
        ends.append((top + torch.log(total)).view(hk, m, rep).transpose(0, 1).reshape(m, hq))
    return {"o": torch.cat(outs).to(q.dtype), "lse": torch.cat(ends)}


def _plain_sample(s):
    # in 64 bits: a cumulative sum next to its border decides for a token
    x = torch.nan_to_num(s["logits"].float(), nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf)
    vocab = x.shape[1]
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t == 0
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(greedy, torch.ones_like(t), t))
    place = torch.arange(vocab, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = torch.where((place < k) | (k == 0), w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        keep = (cum - w < p * cum[:, -1:]) | (p >= 1)
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    mass = torch.where(keep, w, torch.zeros_like(w)).sum(1, keepdim=True)
    at = (cum <= s["u"].double()[:, None] * mass).sum(1, keepdim=True)
    at = torch.where(greedy, torch.zeros_like(at), torch.clamp(at, max=vocab - 1))
    logprob = torch.where(greedy, torch.zeros_like(mass), torch.log(w.gather(1, at) / mass))
    return {"token": order.gather(1, at)[:, 0].to(torch.int32), "logprob": logprob[:, 0].float()}


def _plain_extend(s):
    new, kv, table, ps = s["new"].long(), s["kv"].long(), s["table"], s["case"]["page"]
    n, most = table.shape
    base = kv
    column = torch.arange(most, device=DEV)
    if s["prefix_of"] is not None:
        hit = s["prefix_of"].long()
        base = torch.where(hit >= 0, s["prefix_len"].long()[torch.clamp(hit, min=0)], kv)
        wide = s["prefix_table"].shape[1]
        entry = s["prefix_table"][torch.clamp(hit, min=0)][:, torch.clamp(column, max=wide - 1)]
        table.copy_(torch.where((hit >= 0)[:, None] & (column < (base // ps)[:, None]), entry, table))
    have = (base + ps - 1) // ps
    need = (base + new + ps - 1) // ps - have
    first = s["at"].long() + torch.cumsum(need, 0) - need
    taken = column - have[:, None]
    fresh = (taken >= 0) & (taken < need[:, None])
    table.copy_(torch.where(fresh, s["free"][torch.clamp(first[:, None] + taken, 0, s["free"].numel() - 1)], table))
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    token = torch.arange(s["case"]["tokens"] + 8, device=DEV)
    seq = torch.clamp(torch.searchsorted(cu[1:].contiguous(), token, right=True), max=n - 1)
    live = token < cu[-1]
    pos = base[seq] + token - cu[seq]
    slot = table[seq, torch.clamp(pos // ps, max=most - 1)].long() * ps + pos % ps
    none = torch.full((), -1, device=DEV)
    return {"table": table, "cu": cu.to(torch.int32), "kv": (base + new).to(torch.int32), "at": (s["at"] + need.sum()).to(torch.int32),
            "slots": torch.where(live, slot, none), "positions": torch.where(live, pos, none).to(torch.int32)}


_plain = {"attn": _plain_attn, "sample": _plain_sample, "extend": _plain_extend}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        lens, ps = _attn_sizes(case)[0], case["page"]
        cu, kv, table = _cu(lens), s["kv_len"].tolist(), s["table"].tolist()
        rep, d = case["h_q"] // case["h_kv"], case["d"]
        out, lse = [], []
        for i, n in enumerate(lens):  # every request by itself, over all of its keys
            ids = torch.tensor(table[i][:-(-kv[i] // ps)], device=DEV)
            keys, vals = (c[ids].flatten(0, 1)[:kv[i]].double() for c in (s["kc"], s["vc"]))
            hidden = torch.arange(kv[i], device=DEV)[None] > kv[i] - n + torch.arange(n, device=DEV)[:, None]
            heads, ends = [], []
            for h in range(case["h_q"]):
                score = (s["q"][cu[i]:cu[i + 1], h].double() @ keys[:, h // rep].t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
                ends.append(torch.logsumexp(score, -1))
                heads.append(torch.exp(score - ends[-1][:, None]) @ vals[:, h // rep])
            out.append(torch.stack(heads, 1))
            lse.append(torch.stack(ends, 1))
        return {"o": torch.cat(out), "lse": torch.cat(lse)}
    if case["op"] == "sample":
        tokens, logs = [], []
        for i in range(case["rows"]):  # a row at a time, by probabilities of the whole vocabulary
            x = s["logits"][i].double()
            t = float(s["temperature"][i])
            if t == 0.0:
                tokens.append(int((x == x.max()).nonzero()[0]))
                logs.append(0.0)
                continue
            order = torch.argsort(-x, stable=True)
            p = torch.softmax(x / t, 0)[order]
            k = int(s["top_k"][i]) if s["top_k"] is not None else 0
            if k:
                p = p[:k]
            p = p / p.sum()
            edge = float(s["top_p"][i]) if s["top_p"] is not None else 1.0
            m = p.numel() if edge >= 1.0 else int((torch.cumsum(p, 0) < edge).sum()) + 1
            if s["min_p"] is not None:
                m = min(m, int((p >= p[0] * float(s["min_p"][i])).sum()))
            p = p[:m] / p[:m].sum()
            at = min(int((torch.cumsum(p, 0) <= float(s["u"][i])).sum()), m - 1)
            tokens.append(int(order[at]))
            logs.append(float(torch.log(p[at])))
        return {"token": torch.tensor(tokens, dtype=torch.int32, device=DEV), "logprob": torch.tensor(logs, dtype=torch.float64, device=DEV)}
    lens, old, hit, pre = _extend_sizes(case)
    ps, table, free = case["page"], s["table"].tolist(), s["free"].tolist()
    at, cu, kv, slots, positions = 7, [0], [], [], []
    for i, n in enumerate(lens):  # a request at a time, a token at a time
        base = old[i]
        if hit[i] >= 0:
            base = pre[hit[i]]
            table[i][:base // ps] = s["prefix_table"][hit[i], :base // ps].tolist()
        for pos in range(base, base + n):
            if pos % ps == 0:
                table[i][pos // ps] = free[at]
                at += 1
            slots.append(table[i][pos // ps] * ps + pos % ps)
            positions.append(pos)
        cu.append(cu[-1] + n)
        kv.append(base + n)
    rest = [-1] * (case["tokens"] + 8 - len(slots))

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=DEV)

    return {"table": ints(table), "cu": ints(cu), "kv": ints(kv), "at": ints([at]), "slots": ints(slots + rest, torch.int64), "positions": ints(positions + rest)}
