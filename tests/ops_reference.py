"""Plain 64-bit implementations of the suffix and decode operators, one token at a time, for the
tests (float64 on the CPU).  Each also returns the sum of absolute values behind every result
element ("abs"), which the tolerances are multiples of: a computation whose roundings are each at
most u relative is off by at most (their number along the longest path) u times that sum."""
from __future__ import annotations

import math

import torch

U32 = torch.finfo(torch.float32).eps / 2          # half a step of fp32


def u(dtype) -> float:
    """Half a step of a type, relative to the value: one rounding."""
    return torch.finfo(dtype).eps / 2


def d(t):
    return t.detach().cpu().double()


def conv_tokens(x, weight, bias, state, silu):
    """x [L, C], state [W - 1, C] -> y [L, C], abs, state behind."""
    W = weight.shape[1]
    rows = torch.cat([state, x])
    y, ab = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        win = rows[t:t + W].t()
        y[t] = (win * weight).sum(1)
        ab[t] = (win * weight).abs().sum(1)
    if bias is not None:
        y, ab = y + bias, ab + bias.abs()
    return (y * torch.sigmoid(y) if silu else y), ab, rows[rows.shape[0] - (W - 1):]


def ssm_tokens(x, B, C, dt, A, D, dt_bias, S, softplus=True):
    """x [L, H, P], B, C [L, G, N], dt [L, H], S [H, N, P] -> y, y abs, S, S abs."""
    rep = x.shape[1] // B.shape[1]
    B, C = B.repeat_interleave(rep, 1), C.repeat_interleave(rep, 1)
    if dt_bias is not None:
        dt = dt + dt_bias
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros((), dtype=torch.float64))
    S, Sa = S.clone(), S.abs()
    y, ya = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        a = torch.exp(dt[t] * A)[:, None, None]
        w = B[t][:, :, None] * (dt[t][:, None] * x[t])[:, None, :]
        S, Sa = a * S + w, a * Sa + w.abs()
        y[t], ya[t] = (S * C[t][:, :, None]).sum(1), (Sa * C[t][:, :, None].abs()).sum(1)
        if D is not None:
            y[t] += D[:, None] * x[t]
            ya[t] += (D[:, None] * x[t]).abs()
    return y, ya, S, Sa


def delta_token(q, k, v, g, beta, S, scale):
    """One token of one row: q, k [G, N], v [H, P], g, beta [H], S [H, N, P] -> o, o abs, S, S abs."""
    rep = v.shape[0] // q.shape[0]
    q, k = q.repeat_interleave(rep, 0), k.repeat_interleave(rep, 0)
    a = torch.exp(g)[:, None, None]
    p = (a * S * k[:, :, None]).sum(1)
    pa = (a * S * k[:, :, None]).abs().sum(1)
    un, ua = beta[:, None] * (v - p), beta[:, None].abs() * (v.abs() + pa)
    new, na = a * S + k[:, :, None] * un[:, None, :], (a * S).abs() + k[:, :, None].abs() * ua[:, None, :]
    o, oa = scale * (new * q[:, :, None]).sum(1), abs(scale) * (na * q[:, :, None].abs()).sum(1)
    return o, oa, new, na


def rope_head(x, weight, eps, norm, cos, sin, interleaved):
    """x [..., d], cos, sin [r] -> rotated, abs (the two products of a pair)."""
    y = x
    if norm:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight
    r = cos.numel()
    out, ab = y.clone(), y.abs()
    for i in range(r):
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        a, b = y[..., i0], y[..., i1]
        out[..., i0], out[..., i1] = a * cos[i] - b * sin[i], b * cos[i] + a * sin[i]
        ab[..., i0] = (a * cos[i]).abs() + (b * sin[i]).abs()
        ab[..., i1] = (b * cos[i]).abs() + (a * sin[i]).abs()
    return out, ab


def attend(q, keys, vals, pos, scale):
    """q [H, d] at position pos, keys and vals [kv, K, d] -> o, o abs, lse, largest sum |scale q k|."""
    H, dim = q.shape
    rep = H // keys.shape[1]
    n = max(0, min(pos + 1, keys.shape[0]))
    o, oa = torch.zeros(H, dim, dtype=torch.float64), torch.zeros(H, dim, dtype=torch.float64)
    lse, big = torch.full((H,), -math.inf, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    if n == 0:
        return o, oa, lse, big
    for h in range(H):
        kh, vh = keys[:n, h // rep], vals[:n, h // rep]
        s = scale * (kh @ q[h])
        lse[h] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[h])
        o[h], oa[h] = p @ vh, p @ vh.abs()
        big[h] = abs(scale) * (kh.abs() @ q[h].abs()).max()
    return o, oa, lse, big


def within(got, want, tol, what):
    """Every element at most its tolerance off; says the worst one."""
    err = (d(got) - want).abs()
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(err)
    bad = ~(err <= tol)
    if bad.any():
        i = int(torch.where(bad, err / tol.clamp(min=1e-300), torch.zeros(())).argmax())
        raise AssertionError("%s: %d of %d off; worst at %d: got %r, want %r, tolerance %.3g" % (
            what, int(bad.sum()), bad.numel(), i, float(d(got).reshape(-1)[i]), float(want.reshape(-1)[i]),
            float(tol.reshape(-1)[i])))
