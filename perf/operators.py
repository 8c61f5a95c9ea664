"""Operators of a hybrid model's suffix and decode steps: their workloads, plain forms and exact values.

After a prefix-cache hit a hybrid model prefills the unmatched suffix and then produces tokens
one by one.  Beside the gated delta rule's prefill that takes a short causal convolution, a
selective state space scan, single-token steps of both recurrences, the norm and rotation of q
and k with the append to a paged cache, and the attention of the new tokens over that cache.
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
        # the q, k and v channels of one linear layer (16 q/k heads, 32 v heads, 128 each): the
        # prompts of a packed batch of unmatched suffixes, continued from the matched prefixes
        dict(name="conv_suffixes", op="conv", dtype="bf16", channels=8192, width=4, n_seqs=16, tokens=8200, lens=1, start=True),
        # the same layer's next token of 64 requests, fp32
        dict(name="conv_next_token", op="conv_step", dtype="f32", channels=8192, width=4, rows=64, slots=80),
        # a whole 32K prompt of one sequence through one state space layer: few chains, long
        dict(name="scan_long_prompt", op="scan", dtype="bf16", groups=2, heads=32, d_k=128, d_v=64, n_seqs=1, tokens=32768, lens=0, start=False),
        # many short prompts of different lengths, continued from their states, fp32
        dict(name="scan_packed_f32", op="scan", dtype="f32", groups=4, heads=4, d_k=64, d_v=64, n_seqs=24, tokens=7001, lens=2, start=True),
        # the next token of 64 requests, one state space layer
        dict(name="ssm_next_token", op="ssm_step", dtype="bf16", groups=2, heads=32, d_k=128, d_v=64, rows=64, slots=96),
        # the next token of 48 requests, one gated delta layer (16 q/k heads, 32 v heads)
        dict(name="delta_next_token", op="delta_step", dtype="bf16", groups=16, heads=32, d_k=128, d_v=128, rows=48, slots=48),
        # a 1024-token suffix behind a 31744-token hit, one attention layer (2 KV heads of 256)
        dict(name="rope_suffix", op="rope", dtype="bf16", h_q=16, h_kv=2, d=256, rot=64, page=64, n_seqs=1, tokens=1024, lens=0, context=31744, interleaved=False),
        # the next token of 33 requests, every dimension rotated in neighbouring pairs, fp32
        dict(name="rope_next_token", op="rope", dtype="f32", h_q=8, h_kv=4, d=128, rot=128, page=16, n_seqs=33, tokens=33, lens=0, context=3000, interleaved=True),
        # the next token of one request: the smallest call
        dict(name="attn_one_token", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=16, n_seqs=1, tokens=1, lens=0, context=8191),
        # the next token of 64 requests with contexts of 1K to 32K
        dict(name="attn_next_token", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=64, n_seqs=64, tokens=64, lens=0, context=32768),
        # a 1024-token suffix behind a 31744-token hit
        dict(name="attn_suffix", op="attn", dtype="bf16", h_q=16, h_kv=2, d=256, page=64, n_seqs=1, tokens=1024, lens=0, context=31744),
        # suffixes of different lengths behind different hits, fp32
        dict(name="attn_packed_f32", op="attn", dtype="f32", h_q=16, h_kv=4, d=64, page=24, n_seqs=9, tokens=1501, lens=3, context=4000),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["conv", "conv_step", "scan", "scan", "ssm_step", "delta_step", "rope", "attn", "attn", "attn"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    half = 2 if c["dtype"] == "f32" else 1
    if op in ("conv", "conv_step"):
        c.update(channels=8 * log(16, 1024 // half), width=rng.choice([2, 3, 4, 4]))
        if op == "conv":
            c.update(n_seqs=log(1, 64), tokens=log(1, 8200), lens=rng.randrange(1, 1000), start=rng.random() < 0.5)
        else:
            c.update(rows=log(1, 300))
            c.update(slots=c["rows"] + rng.randrange(0, 40))
    elif op == "scan":
        g = rng.choice([1, 2, 4])
        c.update(groups=g, heads=g * rng.choice([1, 2, 4, 8]), d_k=rng.choice([64, 128]), d_v=rng.choice([64, 128]))
        c.update(n_seqs=log(1, 40), tokens=log(1, 8192 // half), lens=rng.randrange(1, 1000), start=rng.random() < 0.5)
    elif op in ("ssm_step", "delta_step"):
        g = rng.choice([1, 2, 4, 8, 16])
        c.update(groups=g, heads=g * rng.choice([1, 2, 4]), d_k=rng.choice([64, 128]), d_v=rng.choice([64, 128]), rows=log(1, 128))
        c.update(slots=c["rows"] + rng.randrange(0, 40))
    else:
        kv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128, 256])
        c.update(h_q=kv * rng.choice([1, 2, 3, 4, 8]), h_kv=kv, d=d, page=rng.choice([1, 16, 24, 32, 64, 128, 256]), n_seqs=log(1, 64))
        c.update(tokens=rng.choice([c["n_seqs"], c["n_seqs"] + log(1, 1000)]), lens=rng.randrange(1, 1000), context=log(1, 16384 // half))
        if op == "rope":
            c.update(rot=rng.choice([0, d // 4, d // 2, d]), interleaved=rng.random() < 0.3)
        else:  # no dearer than the suffix behind the 32K hit
            while c["tokens"] * c["context"] * c["h_q"] * d * half > 1024 * 31744 * 16 * 256 // 4 or c["n_seqs"] * c["context"] * kv * d * half > 64 * 16384 * 512:
                c["context"] = max(1, c["context"] // 2)
                c["tokens"] = max(c["n_seqs"], c["tokens"] * 3 // 4)
                c["n_seqs"] = min(c["n_seqs"], c["tokens"])
    return c


# ------------------------------------------------------------------ lengths
def _lens(case):
    """Tokens of each packed sequence: equal shares (lens = 0), or spread unevenly, some of them empty."""
    n, t = case["n_seqs"], case["tokens"]
    if case["lens"] == 0:
        return [t // n + (1 if i < t % n else 0) for i in range(n)]
    r = random.Random(case["lens"] * 7919 + n)
    if t == n:
        return [1] * n
    w = [r.random() ** 2 if r.random() > 0.1 else 0.0 for _ in range(n)]
    s = sum(w) or 1.0
    got = [int(t * x / s) for x in w]
    got[r.randrange(n)] += t - sum(got)
    return got


def _contexts(case):
    """Tokens that each sequence has in the cache before the new ones."""
    n, c = case["n_seqs"], case["context"]
    if n == 1:
        return [c]
    r = random.Random(case["lens"] * 104729 + n + c)
    return [r.randrange(min(c, max(0, c // 32)), c + 1) for _ in range(n)]


def _cu(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return at


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, dt = case["op"], _DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = {"case": dict(case)}
    if own:
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)  # a caller keeps its workspace
    if op in ("conv", "conv_step"):
        ch, w = case["channels"], case["width"]
        rows = case["tokens"] if op == "conv" else case["rows"]
        s["x"] = normal(rows, ch)
        s["weight"] = uniform(ch, w, lo=-1.0, hi=1.0) / w ** 0.5
        s["bias"] = normal(ch, scale=0.1, dtype=torch.float32)
        if op == "conv":
            s["cu"] = ints(_cu(_lens(case)))
            s["state0"] = normal(case["n_seqs"], w - 1, ch) if case["start"] else None
        else:
            s["state"] = normal(case["slots"], w - 1, ch)
            s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:rows].to(torch.int32)
    elif op in ("scan", "ssm_step"):
        h, k, p, gr = case["heads"], case["d_k"], case["d_v"], case["groups"]
        rows = case["tokens"] if op == "scan" else case["rows"]
        # x, B, C and dt are columns of one projection's output
        wide = h * p + 2 * gr * k + 8 * ((h + 7) // 8)
        buf = normal(rows, wide)
        s["x"] = buf[:, :h * p].unflatten(1, (h, p))
        s["B"] = buf[:, h * p:h * p + gr * k].unflatten(1, (gr, k))
        s["C"] = buf[:, h * p + gr * k:h * p + 2 * gr * k].unflatten(1, (gr, k))
        s["dt"] = buf[:, h * p + 2 * gr * k:h * p + 2 * gr * k + h]
        s["A"] = -uniform(h, lo=1.0, hi=16.0)
        s["D"] = normal(h, dtype=torch.float32)
        step = torch.exp(uniform(h, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        if op == "scan":
            s["cu"] = ints(_cu(_lens(case)))
            s["S0"] = normal(case["n_seqs"], h, k, p, dtype=torch.float32) if case["start"] else None
            if own:
                import gated_deltanet_state_gdn_amd as gdn
                desc = gdn.make_ssm_desc(s["x"], s["B"], case["n_seqs"])
                s["ws"] = torch.zeros(gdn.gdn_ssm_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
        else:
            s["S"] = normal(case["slots"], h, k, p, dtype=torch.float32)
            s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:rows].to(torch.int32)
    elif op == "delta_step":
        h, k, p, gr, rows = case["heads"], case["d_k"], case["d_v"], case["groups"], case["rows"]
        unit = [normal(rows, gr, k, dtype=torch.float32) for _ in range(2)]
        s["q"], s["k"] = [(u / u.norm(dim=-1, keepdim=True)).to(dt) for u in unit]
        s["v"] = normal(rows, h, p)
        s["g"] = -torch.nn.functional.softplus(normal(rows, h, dtype=torch.float32) - 4.0)
        s["beta"] = torch.sigmoid(normal(rows, h, dtype=torch.float32))
        s["S"] = normal(case["slots"], h, k, p, scale=0.3, dtype=torch.float32)
        s["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:rows].to(torch.int32)
    else:
        lens, ctx = _lens(case), _contexts(case)
        total = [a + b for a, b in zip(lens, ctx)]
        hq, hk, d, ps = case["h_q"], case["h_kv"], case["d"], case["page"]
        per = [-(-x // ps) for x in total]
        pages = sum(per) + 3
        order = torch.randperm(pages, generator=g, device=DEV)[:sum(per)].to(torch.int32)
        table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32, device=DEV)
        at = torch.arange(table.shape[1], device=DEV)[None] < torch.tensor(per, device=DEV)[:, None]
        table[at] = order
        s.update(table=table, cu=ints(_cu(lens)), kv_len=ints(total), longest=max(total), most=max(lens))
        s["kc"], s["vc"] = normal(pages, ps, hk, d), normal(pages, ps, hk, d)
        s["q"] = normal(case["tokens"], hq, d)
        if op == "rope":
            s["k"], s["v"] = normal(case["tokens"], hk, d), normal(case["tokens"], hk, d)
            s["wq"], s["wk"] = uniform(d, lo=0.5, hi=1.5), uniform(d, lo=0.5, hi=1.5)
            rot = case["rot"]
            f = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))
            a = torch.arange(max(max(total), 1), device=DEV, dtype=torch.float64)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        elif own:
            import gated_deltanet_state_gdn_amd as gdn
            desc = gdn.make_paged_desc(s["q"], s["kc"], s["table"], len(lens), max_kv_len=s["longest"])
            s["ws"] = torch.zeros(gdn.gdn_paged_workspace_bytes(desc), dtype=torch.uint8, device=DEV)
    return s


def work(case):
    op, e = case["op"], _BYTES[case["dtype"]]
    if op in ("conv", "conv_step"):
        ch, w = case["channels"], case["width"]
        rows = case["tokens"] if op == "conv" else case["rows"]
        states = (case["n_seqs"] * (2 if case["start"] else 1)) if op == "conv" else 2 * rows
        return {"bytes": 2 * rows * ch * e + states * (w - 1) * ch * e + ch * (w + 1) * 4, "flops": 2 * w * rows * ch}
    if op in ("scan", "ssm_step", "delta_step"):
        h, k, p, gr = case["heads"], case["d_k"], case["d_v"], case["groups"]
        rows = case["tokens"] if op == "scan" else case["rows"]
        states = (case["n_seqs"] * (2 if case["start"] else 1)) if op == "scan" else 2 * rows
        gates = 8 if op == "delta_step" else e
        return {"bytes": rows * (2 * h * p * e + 2 * gr * k * e + h * gates) + states * h * k * p * 4, "flops": rows * h * k * p * (6 if op == "delta_step" else 4)}
    lens, ctx = _lens(case), _contexts(case)
    t, hq, hk, d = case["tokens"], case["h_q"], case["h_kv"], case["d"]
    if op == "rope":
        return {"bytes": t * (2 * hq + 4 * hk) * d * e + t * case["rot"] * 4, "flops": t * (hq + hk) * (4 * d + 3 * case["rot"])}
    keys = sum(a + b for a, b in zip(lens, ctx) if a)
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(lens, ctx))
    return {"bytes": 2 * keys * hk * d * e + 2 * t * hq * d * e + t * hq * 4, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_conv(s):
    import gated_deltanet_state_gdn_amd as gdn
    y, state = gdn.gdn_conv(s["x"], s["weight"], s["cu"], bias=s["bias"], state0=s["state0"], ws=s["ws"])
    return {"y": y, "state": state}


def _own_conv_step(s):
    import gated_deltanet_state_gdn_amd as gdn
    y = gdn.gdn_conv_step(s["x"], s["weight"], s["state"], slots=s["slots"], bias=s["bias"], ws=s["ws"])
    return {"y": y, "state": s["state"]}


def _own_scan(s):
    import gated_deltanet_state_gdn_amd as gdn
    S, y, _ = gdn.gdn_ssm_scan(s["x"], s["B"], s["C"], s["dt"], s["A"], s["cu"], D=s["D"], dt_bias=s["dt_bias"], S0=s["S0"], ws=s["ws"])
    return {"S": S, "y": y}


def _own_ssm_step(s):
    import gated_deltanet_state_gdn_amd as gdn
    y = gdn.gdn_ssm_step(s["x"], s["B"], s["C"], s["dt"], s["A"], s["S"], slots=s["slots"], D=s["D"], dt_bias=s["dt_bias"], ws=s["ws"])
    return {"S": s["S"], "y": y}


def _own_delta_step(s):
    import gated_deltanet_state_gdn_amd as gdn
    o = gdn.gdn_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], slots=s["slots"], ws=s["ws"])
    return {"S": s["S"], "o": o}


def _own_rope(s):
    import gated_deltanet_state_gdn_amd as gdn
    q = gdn.gdn_qk_norm_rope(s["q"], s["k"], s["v"], s["cos_sin"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_len"],
                             q_weight=s["wq"], k_weight=s["wk"], interleaved=s["case"]["interleaved"], ws=s["ws"])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _own_attn(s):
    import gated_deltanet_state_gdn_amd as gdn
    o, lse = gdn.gdn_paged_attn(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_len"], max_kv_len=s["longest"], lse=True, ws=s["ws"])
    return {"o": o, "lse": lse}


_own = {"conv": _own_conv, "conv_step": _own_conv_step, "scan": _own_scan, "ssm_step": _own_ssm_step, "delta_step": _own_delta_step, "rope": _own_rope, "attn": _own_attn}


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _sequence_of(cu, tokens):
    """The sequence that each packed token belongs to."""
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=cu.device, dtype=cu.dtype), right=True)


def _plain_conv(s):
    x, w, cu = s["x"], s["weight"], s["cu"].long()
    t, ch = x.shape
    n, k = cu.numel() - 1, w.shape[1]
    # every sequence's old inputs in front of its new ones
    rows = torch.arange(t, device=DEV) + (_sequence_of(cu, t) + 1) * (k - 1)
    seq = torch.arange(n, device=DEV)
    ext = torch.zeros(t + n * (k - 1), ch, device=DEV)
    ext[rows] = x.float()
    if s["state0"] is not None:
        ext[(cu[:-1] + seq * (k - 1))[:, None] + torch.arange(k - 1, device=DEV)] = s["state0"].float()
    y = (ext[rows[:, None] + torch.arange(1 - k, 1, device=DEV)] * w.t()).sum(1) + s["bias"]
    last = (cu[1:] + (seq + 1) * (k - 1))[:, None] + torch.arange(1 - k, 0, device=DEV)
    return {"y": _silu(y).to(x.dtype), "state": ext[last].to(x.dtype)}


def _plain_conv_step(s):
    at = s["slots"].long()
    win = torch.cat([s["state"][at], s["x"][:, None]], 1)
    y = (win.float() * s["weight"].t()).sum(1) + s["bias"]
    s["state"][at] = win[:, 1:]
    return {"y": _silu(y).to(s["x"].dtype), "state": s["state"]}


def _plain_scan(s):
    x, B, C, cu = s["x"], s["B"], s["C"], s["cu"].long()
    t, h, p = x.shape
    gr, k = B.shape[1:]
    n, q = cu.numel() - 1, 64
    longest = max(_lens(s["case"]))
    nc = max(1, -(-longest // q))
    # [sequence, chunk, token in chunk], zeros behind each sequence's end
    at = cu[:-1, None] + torch.arange(nc * q, device=DEV)
    live = (at < cu[1:, None]).view(n, nc, q, 1)
    at = torch.clamp(at, max=max(t - 1, 0)).view(n, nc, q)
    dt = torch.where(live, _softplus(s["dt"].float() + s["dt_bias"])[at], torch.zeros((), device=DEV))
    xs = torch.where(live[..., None], x[at].float(), torch.zeros((), device=DEV)).transpose(2, 3)
    Bs = torch.where(live[..., None], B[at].float(), torch.zeros((), device=DEV)).transpose(2, 3)
    Cs = torch.where(live[..., None], C[at].float(), torch.zeros((), device=DEV)).transpose(2, 3)
    G = torch.cumsum((dt.double() * s["A"]), 2).transpose(2, 3)  # [n, nc, h, q]
    dth = dt.transpose(2, 3)
    low = torch.ones(q, q, device=DEV, dtype=torch.bool).tril()
    L = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], torch.full((), -math.inf, device=DEV, dtype=torch.float64))).float()
    CB = torch.matmul(Cs, Bs.transpose(-1, -2)).repeat_interleave(h // gr, 2)
    y = torch.matmul(CB * L * dth[..., None, :], xs)
    into = (torch.exp(G[..., -1:] - G).float() * dth)[..., None] * xs
    states = torch.matmul(Bs.repeat_interleave(h // gr, 2).transpose(-1, -2), into)  # [n, nc, h, k, p]
    S0 = s["S0"] if s["S0"] is not None else torch.zeros(n, h, k, p, device=DEV)
    states = torch.cat([S0[:, None], states], 1).permute(0, 2, 1, 3, 4).reshape(n, h, nc + 1, k * p)
    total = torch.nn.functional.pad(torch.cumsum(G[..., -1], 1), (0, 0, 1, 0)).transpose(1, 2)  # [n, h, nc + 1]
    lowc = torch.ones(nc + 1, nc + 1, device=DEV, dtype=torch.bool).tril()
    carry = torch.exp(torch.where(lowc, total[..., :, None] - total[..., None, :], torch.full((), -math.inf, device=DEV, dtype=torch.float64))).float()
    before = torch.matmul(carry, states).view(n, h, nc + 1, k, p)
    Ch = Cs.repeat_interleave(h // gr, 2) * torch.exp(G).float()[..., None]
    y = y + torch.matmul(Ch, before[:, :, :-1].transpose(1, 2)) + s["D"][:, None, None] * xs
    y = y.transpose(2, 3).reshape(n * nc * q, h, p)
    where = torch.arange(t, device=DEV)
    seq = _sequence_of(cu, t)
    return {"S": before[:, :, -1].contiguous(), "y": y[seq * nc * q + where - cu[seq]].to(x.dtype)}


def _plain_ssm_step(s):
    at, rep = s["slots"].long(), s["x"].shape[1] // s["B"].shape[1]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    x = s["x"].float()
    B, C = s["B"].float().repeat_interleave(rep, 1), s["C"].float().repeat_interleave(rep, 1)
    S = torch.exp(dt * s["A"])[..., None, None] * s["S"][at] + B[..., None] * (dt[..., None] * x)[..., None, :]
    s["S"][at] = S
    return {"S": s["S"], "y": ((S * C[..., None]).sum(2) + s["D"][:, None] * x).to(s["x"].dtype)}


def _plain_delta_step(s):
    at, rep = s["slots"].long(), s["v"].shape[1] // s["k"].shape[1]
    q, k = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1)
    S = torch.exp(s["g"])[..., None, None] * s["S"][at]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(2))
    S = S + k[..., None] * u[..., None, :]
    s["S"][at] = S
    return {"S": s["S"], "o": (S * q[..., None]).sum(2).to(s["v"].dtype)}


def _rotated(x, cos_sin, interleaved):
    r = cos_sin.shape[-1] // 2
    c, n = cos_sin[:, None, :r], cos_sin[:, None, r:]
    a, b = (x[..., :2 * r:2], x[..., 1:2 * r:2]) if interleaved else (x[..., :r], x[..., r:2 * r])
    u, v = a * c - b * n, b * c + a * n
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * r:]], -1)


def _plain_rope(s):
    cu, q, k = s["cu"].long(), s["q"].float(), s["k"].float()
    t, ps = q.shape[0], s["kc"].shape[1]
    seq = _sequence_of(cu, t)
    pos = s["kv_len"].long()[seq] - cu[seq + 1] + torch.arange(t, device=DEV)
    turn = s["cos_sin"][pos]
    inter = s["case"]["interleaved"]
    q = _rotated(q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["wq"], turn, inter)
    k = _rotated(k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["wk"], turn, inter)
    page = s["table"][seq, pos // ps].long()
    s["kc"][page, pos % ps] = k.to(s["kc"].dtype)
    s["vc"][page, pos % ps] = s["v"]
    return {"q": q.to(s["q"].dtype), "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_attn(s):
    q, cu, kv = s["q"], s["cu"].long(), s["kv_len"].long()
    t, hq, d = q.shape
    ps, hk = s["kc"].shape[1:3]
    n, most, longest = kv.numel(), s["most"], s["longest"]
    table = torch.clamp(s["table"], min=0).long()
    keys = s["kc"][table].view(n, -1, hk, d)[:, :longest].float().permute(0, 2, 3, 1)
    vals = s["vc"][table].view(n, -1, hk, d)[:, :longest].float().transpose(1, 2)
    at = cu[:-1, None] + torch.arange(most, device=DEV)
    rows = q[torch.clamp(at, max=t - 1)].float().view(n, most, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    pos = (kv - cu[1:])[:, None] + at
    seen = torch.arange(longest, device=DEV) <= pos[..., None]
    seen = seen.repeat_interleave(hq // hk, 1)[:, None]
    score = torch.matmul(rows * d ** -0.5, keys).masked_fill_(~seen, -math.inf)
    top = torch.clamp(score.amax(-1, keepdim=True), min=-1e30)
    score = torch.exp(score.sub_(top))
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, vals) / torch.clamp(total, min=1e-37)
    lse = (top + torch.log(total))[..., 0]
    seq = _sequence_of(cu, t)
    at = seq * most + torch.arange(t, device=DEV) - cu[seq]

    def packed(v):
        return v.view(n, hk, most, hq // hk, -1).permute(0, 2, 1, 3, 4).reshape(n * most, hq, -1)[at]

    return {"o": packed(o).to(q.dtype), "lse": packed(lse)[..., 0].contiguous()}


_plain = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "ssm_step": _plain_ssm_step, "delta_step": _plain_delta_step, "rope": _plain_rope, "attn": _plain_attn}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_step"):
        w, b = s["weight"].double(), s["bias"].double()
        k = w.shape[1]

        def sums(rows):  # [k - 1 + L, channels] -> [L, channels]
            y = b.clone().expand(rows.shape[0] - k + 1, -1)
            for j in range(k):
                y = y + w[:, j] * rows[j:j + y.shape[0]]
            return y * torch.sigmoid(y)

        if op == "conv_step":
            state, out = s["state"].double(), []
            for i, at in enumerate(s["slots"].tolist()):
                rows = torch.cat([state[at], s["x"][i:i + 1].double()])
                out.append(sums(rows))
                state[at] = rows[1:]
            return {"y": torch.cat(out), "state": state}
        out, ends, cu = [], [], s["cu"].tolist()
        for i in range(case["n_seqs"]):
            old = s["state0"][i].double() if s["state0"] is not None else torch.zeros(k - 1, w.shape[0], device=DEV, dtype=torch.float64)
            rows = torch.cat([old, s["x"][cu[i]:cu[i + 1]].double()])
            out.append(sums(rows))
            ends.append(rows[rows.shape[0] - k + 1:])
        return {"y": torch.cat(out), "state": torch.stack(ends)}
    if op in ("scan", "ssm_step"):
        rep = case["heads"] // case["groups"]
        x = s["x"].double()
        B, C = (v.double().repeat_interleave(rep, 1) for v in (s["B"], s["C"]))
        dt = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros((), device=DEV, dtype=torch.float64))
        a = torch.exp(dt * s["A"].double())
        D = s["D"].double()[:, None]

        def token(S, i):  # the rows i of the inputs, one for each state
            S = a[i][..., None, None] * S + B[i][..., None] * (dt[i][..., None] * x[i])[..., None, :]
            return S, torch.matmul(C[i][..., None, :], S)[..., 0, :] + D * x[i]

        if op == "ssm_step":
            at, S = s["slots"].long(), s["S"].double()
            S[at], y = token(S[at], torch.arange(case["rows"], device=DEV))
            return {"S": S, "y": y}
        lens, cu = _lens(case), _cu(_lens(case))
        S = s["S0"].double() if s["S0"] is not None else torch.zeros(case["n_seqs"], case["heads"], case["d_k"], case["d_v"], device=DEV, dtype=torch.float64)
        y = torch.empty(case["tokens"], case["heads"], case["d_v"], device=DEV, dtype=torch.float64)
        by_length = sorted(range(len(lens)), key=lambda i: -lens[i])
        order, first = torch.tensor(by_length, device=DEV), torch.tensor([cu[i] for i in by_length], device=DEV)
        S = S[order]
        live = len(lens)
        for step in range(max(lens)):
            while lens[by_length[live - 1]] <= step:
                live -= 1
            S[:live], y[first[:live] + step] = token(S[:live], first[:live] + step)
        back = torch.empty_like(S)
        back[order] = S
        return {"S": back, "y": y}
    if op == "delta_step":
        at, rep = s["slots"].long(), case["heads"] // case["groups"]
        q, k = (v.double().repeat_interleave(rep, 1) for v in (s["q"], s["k"]))
        old, beta = s["S"].double()[at], s["beta"].double()[..., None, None]
        kk = torch.eye(case["d_k"], device=DEV, dtype=torch.float64) - beta * (k[..., :, None] * k[..., None, :])
        new = torch.exp(s["g"].double())[..., None, None] * torch.matmul(kk, old) + beta * (k[..., :, None] * s["v"].double()[..., None, :])
        S = s["S"].double()
        S[at] = new
        return {"S": S, "o": torch.matmul(q[..., None, :], new)[..., 0, :]}
    lens, cu, kv, ps = _lens(case), _cu(_lens(case)), s["kv_len"].tolist(), case["page"]
    table = s["table"].tolist()
    if op == "rope":
        keys, vals = s["kc"].double(), s["vc"].double()
        at = [(i, kv[i] - n + j) for i, n in enumerate(lens) for j in range(n)]
        pos = torch.tensor([p for _, p in at], device=DEV)
        page = torch.tensor([table[i][p // ps] for i, p in at], device=DEV)
        half = case["rot"] // 2
        turn = s["cos_sin"].double()[pos]
        z = torch.complex(turn[:, :half], turn[:, half:])[:, None]

        def turned(v, w):
            v = v.double()
            v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            head = v[..., :2 * half]
            if case["interleaved"]:
                head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * z).flatten(-2)
            else:
                r = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * z
                head = torch.cat([r.real, r.imag], -1)
            return torch.cat([head, v[..., 2 * half:]], -1)

        q, k = turned(s["q"], s["wq"]), turned(s["k"], s["wk"])
        keys[page, pos % ps], vals[page, pos % ps] = k, s["v"].double()
        return {"q": q, "k_cache": keys, "v_cache": vals}
    hq, hk, d = case["h_q"], case["h_kv"], case["d"]
    out, lse = [], []
    for i, n in enumerate(lens):
        if n == 0:
            continue
        ids = torch.tensor(table[i][:-(-kv[i] // ps)], device=DEV)
        keys, vals = (c[ids].flatten(0, 1)[:kv[i]].double() for c in (s["kc"], s["vc"]))
        pos = kv[i] - n + torch.arange(n, device=DEV)
        hidden = torch.arange(kv[i], device=DEV)[None] > pos[:, None]
        heads, ends = [], []
        for h in range(hq):
            kh, vh = keys[:, h // (hq // hk)], vals[:, h // (hq // hk)]
            score = (s["q"][cu[i]:cu[i + 1], h].double() @ kh.t() / math.sqrt(d)).masked_fill(hidden, -math.inf)
            ends.append(torch.logsumexp(score, -1))
            heads.append(torch.exp(score - ends[-1][:, None]) @ vh)
        out.append(torch.stack(heads, 1))
        lse.append(torch.stack(ends, 1))
    return {"o": torch.cat(out), "lse": torch.cat(lse)}
