"""Plain 64-bit implementations of the operators around a prefix cache, a request or a row at a time, for
the tests (on the CPU).  Attention behind shared prefixes has ops_reference.attend's values: the sharing
is no part of the mathematics."""
from __future__ import annotations

import math

import torch

HIGHEST = torch.finfo(torch.float32).max


def draw(x, u, T=1.0, k=0, p=1.0, mp=0.0):
    """x [vocab], the settings of one row -> (token, logprob, how far u and p are from a border, in mass)."""
    x = x.detach().cpu().float().double().tolist()
    x = [-math.inf if math.isnan(v) else min(v, HIGHEST) for v in x]
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    top = x[order[0]]
    if top == -math.inf:
        return -1, -math.inf, 1.0
    if T == 0.0:
        return order[0], 0.0, 1.0
    w = [math.exp((x[i] - top) / T) if x[i] > -math.inf else 0.0 for i in order]
    if k:
        w = w[:k]
    all_k = math.fsum(w)
    margin = 1.0
    if p < 1.0:
        run, n = 0.0, 0
        for n, v in enumerate(w, 1):
            run += v
            margin = min(margin, abs(run - p * all_k) / all_k)
            if run >= p * all_k:
                break
        w = w[:n]
    if mp > 0.0:
        w = [v for v in w if v >= mp]
    mass = math.fsum(w)
    run, at = 0.0, 0
    for at, v in enumerate(w):
        run += v
        margin = min(margin, abs(run - u * mass) / mass) if at + 1 < len(w) else margin
        if run > u * mass:
            break
    return order[at], math.log(w[at] / mass), margin


def extend(new, kv, table, free, at, ps, total, prefix_of=None, prefix_table=None, prefix_len=None):
    """Lists of whole numbers -> (table, cu, kv, at, slots, positions), a token at a time."""
    table = [list(row) for row in table]
    cu, out, slots, positions = [0], [], [], []
    for n, add in enumerate(new):
        base = kv[n]
        if prefix_of is not None and prefix_of[n] >= 0:
            base = prefix_len[prefix_of[n]]
            table[n][:base // ps] = prefix_table[prefix_of[n]][:base // ps]
        for pos in range(base, base + add):
            if pos % ps == 0:
                table[n][pos // ps] = free[at]
                at += 1
            slots.append(table[n][pos // ps] * ps + pos % ps)
            positions.append(pos)
        cu.append(cu[-1] + add)
        out.append(base + add)
    rest = [-1] * (total - len(slots))
    return table, cu, out, at, slots + rest, positions + rest
