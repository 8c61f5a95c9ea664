"""Python binding of the suffix and decode operators (see include/gdn.h).

As the rest of the package: the functions carry the names of the C entry points and marshal
arguments.  They check what the C side cannot see (dtypes, shapes, strides, devices) and raise
GdnError with the matching status before anything is enqueued.  Missing outputs are allocated
with torch; ``ws`` is a zero-filled uint8 workspace that the caller keeps (one for each stream or
graph that may run at the same time), and a new one is made for a call without it.  Calls run on
torch's current stream of the tensors' device, or on ``stream``.
"""
from __future__ import annotations

import ctypes

import torch


from ._lib import (GDN_BF16, GDN_ERR_ALIGN, GDN_ERR_DTYPE, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_F32, GDN_OK,
                   GdnConvDesc, GdnDesc, GdnError, GdnPagedDesc, GdnSsmDesc, load)

_DT = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_byref = ctypes.byref
_i32, _f32, _u8 = torch.int32, torch.float32, torch.uint8


def _need(ok, code, what):
    if not ok:
        raise GdnError(code, what)


def _code(x, where):
    """The gdn_dtype of the operator's element type, x's."""
    dt = _DT.get(x.dtype)
    if dt is None:
        raise GdnError(GDN_ERR_DTYPE, where + ": float32 or bfloat16 wanted")
    return dt


def _rows(t, shape, dtype, where):
    """Checks a [rows, ...] tensor whose rows are contiguous; returns the elements between rows."""
    if t is None:
        raise GdnError(GDN_ERR_NULL, where)
    if t.dtype is not dtype:
        raise GdnError(GDN_ERR_DTYPE, where + ": dtype %s, not %s" % (t.dtype, dtype))
    if tuple(t.shape) != shape:
        raise GdnError(GDN_ERR_SHAPE, where + ": shape %s, not %s" % (tuple(t.shape), shape))
    st, inner = t.stride(), 1
    for k in range(len(shape) - 1, 0, -1):
        if st[k] != inner and shape[k] != 1:
            raise GdnError(GDN_ERR_ALIGN, where + ": a row must be contiguous")
        inner *= shape[k]
    return st[0] if shape[0] > 1 else inner


def _whole(t, shape, dtype, where, optional=False):
    """Checks a contiguous tensor (None where optional)."""
    if t is None:
        if optional:
            return
        raise GdnError(GDN_ERR_NULL, where)
    if t.dtype is not dtype:
        raise GdnError(GDN_ERR_DTYPE, where + ": dtype %s, not %s" % (t.dtype, dtype))
    if tuple(t.shape) != shape:
        raise GdnError(GDN_ERR_SHAPE, where + ": shape %s, not %s" % (tuple(t.shape), shape))
    if not t.is_contiguous():
        raise GdnError(GDN_ERR_ALIGN, where + ": must be contiguous")


def _device(where, x, *others):
    """The GPU that every tensor of a call is on."""
    dev = x.get_device()
    _need(dev >= 0, GDN_ERR_SHAPE, where + ": tensors must be on a GPU")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise GdnError(GDN_ERR_SHAPE, where + ": tensors on different devices")
    return dev


def _elsewhere(x, stream):
    """Whether the call has to be made inside another stream's or device's context."""
    return stream is not None or (x.is_cuda and x.get_device() != torch.cuda.current_device())


def _context(x, stream):
    # allocations and the workspace's fill belong to the stream of the call
    if stream is None:
        return torch.cuda.device(x.device)
    _need(x.is_cuda and stream.device == x.device, GDN_ERR_SHAPE, "the stream is on another device")
    return torch.cuda.stream(stream)


def _current(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _workspace(ws, need, dev, where):
    if ws is None:
        return torch.zeros(need, dtype=_u8, device=torch.device("cuda", dev))
    if ws.dtype is not _u8 or not ws.is_contiguous() or ws.get_device() != dev:
        raise GdnError(GDN_ERR_SHAPE, where + ": ws must be a contiguous uint8 tensor on the same device")
    return ws


def _p(t):
    return None if t is None else t.data_ptr()


def _check(code, where):
    if code != GDN_OK:
        raise GdnError(code, where)


def _silu(activation):
    _need(activation in ("silu", None), GDN_ERR_SHAPE, "activation: 'silu' or None")
    return int(activation == "silu")


def gdn_conv(x, weight, cu_seqlens, *, bias=None, state0=None, state_out=True, activation="silu", y=None,
             ws=None, stream=None):
    """Short causal convolution of packed prompts: x [T, channels], weight [channels, width] fp32.

    ``state0`` [n_seqs, width - 1, channels]: the inputs in front of each sequence (None: zero);
    ``state_out``: a tensor (may be state0), True (allocate) or None.  Returns (y, state_out or None).
    """
    if _elsewhere(x, stream):
        with _context(x, stream):
            return gdn_conv(x, weight, cu_seqlens, bias=bias, state0=state0, state_out=state_out,
                            activation=activation, y=y, ws=ws)
    lib, w = load(), "gdn_conv"
    dt = _code(x, w)
    _need(x.dim() == 2 and weight.dim() == 2 and cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0, GDN_ERR_SHAPE,
          w + ": x [T, channels], weight [channels, width], cu_seqlens [n_seqs + 1]")
    (T, ch), n, k = x.shape, cu_seqlens.numel() - 1, weight.shape[1]
    xs = _rows(x, (T, ch), x.dtype, w + ": x")
    _whole(weight, (ch, k), _f32, w + ": weight")
    _whole(bias, (ch,), _f32, w + ": bias", True)
    _whole(cu_seqlens, (n + 1,), _i32, w + ": cu_seqlens")
    _whole(state0, (n, k - 1, ch), x.dtype, w + ": state0", True)
    silu = _silu(activation)
    if state_out is True:
        state_out = torch.empty((n, k - 1, ch), dtype=x.dtype, device=x.device) if k > 1 else None
    elif state_out is False:
        state_out = None
    _whole(state_out, (n, k - 1, ch), x.dtype, w + ": state_out", True)
    if y is None:
        y = torch.empty((T, ch), dtype=x.dtype, device=x.device)
    ys = _rows(y, (T, ch), x.dtype, w + ": y")
    dev = _device(w, x, weight, cu_seqlens, bias, state0, state_out, y)
    ws = _workspace(ws, 256, dev, w)
    d = GdnConvDesc(n, 0, ch, k, dt, silu, T, xs, ys)
    _check(lib.gdn_conv(_byref(d), x.data_ptr(), weight.data_ptr(), _p(bias), cu_seqlens.data_ptr(), _p(state0),
                        _p(state_out), y.data_ptr(), ws.data_ptr(), ws.numel(), _current(dev)), w)
    return y, state_out


def gdn_conv_step(x, weight, state, *, slots=None, bias=None, activation="silu", y=None, ws=None, stream=None):
    """One token per row: x [rows, channels]; ``state`` [n_slots, width - 1, channels] is updated in
    place.  ``slots`` [rows] int32: the state of each row, -1 for a padded one (None: state i for row
    i).  Returns y."""
    if _elsewhere(x, stream):
        with _context(x, stream):
            return gdn_conv_step(x, weight, state, slots=slots, bias=bias, activation=activation, y=y, ws=ws)
    lib, w = load(), "gdn_conv_step"
    dt = _code(x, w)
    _need(x.dim() == 2 and weight.dim() == 2 and state.dim() == 3, GDN_ERR_SHAPE,
          w + ": x [rows, channels], weight [channels, width], state [n_slots, width - 1, channels]")
    (n, ch), k, pool = x.shape, weight.shape[1], state.shape[0]
    xs = _rows(x, (n, ch), x.dtype, w + ": x")
    _whole(weight, (ch, k), _f32, w + ": weight")
    _whole(bias, (ch,), _f32, w + ": bias", True)
    _whole(state, (pool, k - 1, ch), x.dtype, w + ": state")
    _whole(slots, (n,), _i32, w + ": slots", True)
    silu = _silu(activation)
    if y is None:
        y = torch.empty((n, ch), dtype=x.dtype, device=x.device)
    ys = _rows(y, (n, ch), x.dtype, w + ": y")
    dev = _device(w, x, weight, state, slots, bias, y)
    ws = _workspace(ws, 256, dev, w)
    d = GdnConvDesc(n, pool, ch, k, dt, silu, n, xs, ys)
    _check(lib.gdn_conv_step(_byref(d), x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(), _p(slots),
                             y.data_ptr(), ws.data_ptr(), ws.numel(), _current(dev)), w)
    return y


def make_ssm_desc(x, B, n_seqs, *, total_out_tokens=None, n_slots=0, softplus=True) -> GdnSsmDesc:
    """Sizes of a state space call (x [T, h_v, d_v], B [T, h_qk, d_k]), for its workspace."""
    _need(x.dim() == 3 and B.dim() == 3, GDN_ERR_SHAPE, "make_ssm_desc: x [T, h_v, d_v], B [T, h_qk, d_k]")
    T, h, p = x.shape
    g, k = B.shape[1:]
    return GdnSsmDesc(int(n_seqs), int(n_slots), g, h, k, p, _code(x, "make_ssm_desc"), int(bool(softplus)), T,
                      T if total_out_tokens is None else int(total_out_tokens), h * p, g * k, g * k, h, h * p)


def gdn_ssm_workspace_bytes(desc: GdnSsmDesc) -> int:
    return int(load().gdn_ssm_workspace_bytes(_byref(desc)))


def _ssm_inputs(w, x, B, C, dt, A, D, dt_bias, n_seqs, n_slots, out_tokens, softplus):
    d = make_ssm_desc(x, B, n_seqs, total_out_tokens=out_tokens, n_slots=n_slots, softplus=softplus)
    (T, h, p), e = x.shape, x.dtype
    d.x_stride = _rows(x, (T, h, p), e, w + ": x")
    d.b_stride = _rows(B, (T, d.h_qk, d.d_k), e, w + ": B")
    d.c_stride = _rows(C, (T, d.h_qk, d.d_k), e, w + ": C")
    d.dt_stride = _rows(dt, (T, h), e, w + ": dt")
    _whole(A, (h,), _f32, w + ": A")
    _whole(D, (h,), _f32, w + ": D", True)
    _whole(dt_bias, (h,), _f32, w + ": dt_bias", True)
    return d


def gdn_ssm_scan(x, B, C, dt, A, cu_seqlens, *, D=None, dt_bias=None, softplus=True, r=None, total_out_tokens=None,
                 S0=None, S_out=None, y_out=True, cu_out=None, ws=None, stream=None):
    """Selective state space scan of packed prompts: x [T, h_v, d_v], B, C [T, h_qk, d_k], dt [T, h_v].

    ``r`` [n_seqs] int32: only the last r[n] tokens of each sequence (then ``total_out_tokens`` = their
    sum, y packed per window, ``cu_out`` as for gdn_replay).  ``S0`` [n_seqs, h_v, d_k, d_v]: the states
    to start from; ``S_out`` may be S0.  ``y_out``: a tensor, True (allocate) or None.  ``ws``, when
    given, holds gdn_ssm_workspace_bytes(make_ssm_desc(...)) bytes.  Returns (S_out, y or None, cu_out).
    """
    if _elsewhere(x, stream):
        with _context(x, stream):
            return gdn_ssm_scan(x, B, C, dt, A, cu_seqlens, D=D, dt_bias=dt_bias, softplus=softplus, r=r,
                                total_out_tokens=total_out_tokens, S0=S0, S_out=S_out, y_out=y_out,
                                cu_out=cu_out, ws=ws)
    lib, w = load(), "gdn_ssm_scan"
    _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0, GDN_ERR_SHAPE, w + ": cu_seqlens [n_seqs + 1]")
    _need(r is None or total_out_tokens is not None, GDN_ERR_SHAPE, w + ": r needs total_out_tokens")
    n = cu_seqlens.numel() - 1
    d = _ssm_inputs(w, x, B, C, dt, A, D, dt_bias, n, 0, total_out_tokens, softplus)
    shape = (n, d.h_v, d.d_k, d.d_v)
    _whole(cu_seqlens, (n + 1,), _i32, w + ": cu_seqlens")
    _whole(r, (n,), _i32, w + ": r", True)
    _whole(cu_out, (n + 1,), _i32, w + ": cu_out", True)
    _whole(S0, shape, _f32, w + ": S0", True)
    if S_out is None:
        S_out = torch.empty(shape, dtype=_f32, device=x.device)
    _whole(S_out, shape, _f32, w + ": S_out")
    rows = (int(d.total_out_tokens), d.h_v, d.d_v)
    if y_out is True:
        y_out = torch.empty(rows, dtype=x.dtype, device=x.device)
    elif y_out is False:
        y_out = None
    if y_out is not None:
        d.y_stride = _rows(y_out, rows, x.dtype, w + ": y_out")
    dev = _device(w, x, B, C, dt, A, D, dt_bias, cu_seqlens, r, cu_out, S0, S_out, y_out)
    if ws is None:
        ws = _workspace(None, max(256, gdn_ssm_workspace_bytes(d)), dev, w)
    else:
        _workspace(ws, 0, dev, w)
    _check(lib.gdn_ssm_scan(_byref(d), x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A.data_ptr(),
                            _p(dt_bias), _p(D), cu_seqlens.data_ptr(), _p(r), _p(S0), S_out.data_ptr(), _p(y_out),
                            _p(cu_out), ws.data_ptr(), ws.numel(), _current(dev)), w)
    return S_out, y_out, cu_out


def gdn_ssm_step(x, B, C, dt, A, S, *, slots=None, D=None, dt_bias=None, softplus=True, y=None, ws=None, stream=None):
    """One token per row of the state space recurrence; ``S`` [n_slots, h_v, d_k, d_v] is updated in
    place, ``slots`` as for gdn_conv_step.  Returns y [rows, h_v, d_v]."""
    if _elsewhere(x, stream):
        with _context(x, stream):
            return gdn_ssm_step(x, B, C, dt, A, S, slots=slots, D=D, dt_bias=dt_bias, softplus=softplus, y=y, ws=ws)
    lib, w = load(), "gdn_ssm_step"
    _need(S.dim() == 4, GDN_ERR_SHAPE, w + ": S [n_slots, h_v, d_k, d_v]")
    n, pool = x.shape[0], S.shape[0]
    d = _ssm_inputs(w, x, B, C, dt, A, D, dt_bias, n, pool, None, softplus)
    _whole(S, (pool, d.h_v, d.d_k, d.d_v), _f32, w + ": S")
    _whole(slots, (n,), _i32, w + ": slots", True)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    d.y_stride = _rows(y, tuple(x.shape), x.dtype, w + ": y")
    dev = _device(w, x, B, C, dt, A, D, dt_bias, S, slots, y)
    ws = _workspace(ws, 256, dev, w)
    _check(lib.gdn_ssm_step(_byref(d), x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), A.data_ptr(),
                            _p(dt_bias), _p(D), S.data_ptr(), _p(slots), y.data_ptr(), ws.data_ptr(), ws.numel(),
                            _current(dev)), w)
    return y


def gdn_step(q, k, v, g, beta, S, *, slots=None, o=None, scale: float = 1.0, o_dtype=None, ws=None, stream=None):
    """One token per row of the gated delta rule: q, k [rows, h_qk, d_k], v [rows, h_v, d_v], g, beta
    [rows, h_v] fp32; ``S`` [n_slots, h_v, d_k, d_v] is updated in place, ``slots`` as for
    gdn_conv_step.  Returns o [rows, h_v, d_v]."""
    if _elsewhere(q, stream):
        with _context(q, stream):
            return gdn_step(q, k, v, g, beta, S, slots=slots, o=o, scale=scale, o_dtype=o_dtype, ws=ws)
    lib, w = load(), "gdn_step"
    dt = _code(q, w)
    _need(q.dim() == 3 and v.dim() == 3 and S.dim() == 4, GDN_ERR_SHAPE,
          w + ": q, k [rows, h_qk, d_k], v [rows, h_v, d_v], S [n_slots, h_v, d_k, d_v]")
    (n, hq, dk), (h, dv), pool = q.shape, v.shape[1:], S.shape[0]
    _whole(q, (n, hq, dk), q.dtype, w + ": q")
    _whole(k, (n, hq, dk), q.dtype, w + ": k")
    _whole(v, (n, h, dv), q.dtype, w + ": v")
    _whole(g, (n, h), _f32, w + ": g")
    _whole(beta, (n, h), _f32, w + ": beta")
    _whole(S, (pool, h, dk, dv), _f32, w + ": S")
    _whole(slots, (n,), _i32, w + ": slots", True)
    odt = o.dtype if o is not None else o_dtype if o_dtype is not None else q.dtype
    if o is None:
        o = torch.empty((n, h, dv), dtype=odt, device=q.device)
    _whole(o, (n, h, dv), odt, w + ": o")
    dev = _device(w, q, k, v, g, beta, S, slots, o)
    ws = _workspace(ws, 256, dev, w)
    d = GdnDesc(n, hq, h, dk, dv, dt, _DT.get(odt, -1), float(scale), n, n)
    _check(lib.gdn_step(_byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                        S.data_ptr(), pool, _p(slots), o.data_ptr(), ws.data_ptr(), ws.numel(), _current(dev)), w)
    return o


def _paged(w, q, k_cache, v_cache, block_table, n_seqs, max_kv_len):
    dt = _code(q, w)
    _need(q.dim() == 3 and k_cache.dim() == 4 and block_table.dim() == 2, GDN_ERR_SHAPE,
          w + ": q [T, h_q, d], caches [n_pages, page_size, h_kv, d], block_table [n_seqs, max_pages]")
    (T, h, dim), (pages, ps, hk, dk) = q.shape, k_cache.shape
    _need(dk == dim, GDN_ERR_SHAPE, w + ": the caches' head dim is not q's")
    most = block_table.shape[1]
    st = k_cache.stride()
    if v_cache is not None:
        _need(v_cache.shape == k_cache.shape and v_cache.stride() == st, GDN_ERR_SHAPE,
              w + ": k_cache and v_cache differ in shape or strides")
        _need(k_cache.dtype is q.dtype and v_cache.dtype is q.dtype, GDN_ERR_DTYPE, w + ": the caches have q's dtype")
    _need(st[3] == 1, GDN_ERR_ALIGN, w + ": a head's cache entries must be contiguous")
    # strides of dimensions of one element say nothing
    token = st[1] if ps > 1 else max(st[1], dim)
    head = st[2] if hk > 1 else max(st[2], dim)
    if max_kv_len is None:
        max_kv_len = min(most * ps, 1 << 30)
    return GdnPagedDesc(n_seqs=n_seqs, h_q=h, h_kv=hk, d=dim, dtype=dt, page_size=ps, n_pages=pages, max_pages=most,
                        max_kv_len=min(int(max_kv_len), most * ps), scale=dim ** -0.5, total_tokens=T, q_stride=h * dim,
                        k_stride=hk * dim, v_stride=hk * dim, o_stride=h * dim, page_stride=st[0], token_stride=token,
                        head_stride=head)


def make_paged_desc(q, k_cache, block_table, n_seqs, *, max_kv_len=None) -> GdnPagedDesc:
    """Sizes of a paged call, for gdn_paged_attn's workspace.  ``max_kv_len``: the largest kv_len
    that will be passed (None: all that the block table holds)."""
    return _paged("make_paged_desc", q, k_cache, None, block_table, int(n_seqs), max_kv_len)


def gdn_paged_workspace_bytes(desc: GdnPagedDesc) -> int:
    return int(load().gdn_paged_workspace_bytes(_byref(desc)))


def _paged_lists(w, block_table, cu_seqlens, kv_len):
    _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0 and block_table.dim() == 2, GDN_ERR_SHAPE,
          w + ": cu_seqlens [n_seqs + 1], block_table [n_seqs, max_pages]")
    n = cu_seqlens.numel() - 1
    _whole(cu_seqlens, (n + 1,), _i32, w + ": cu_seqlens")
    _whole(kv_len, (n,), _i32, w + ": kv_len")
    _whole(block_table, (n, block_table.shape[1]), _i32, w + ": block_table")
    return n


def gdn_qk_norm_rope(q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len, *, q_weight=None,
                     k_weight=None, eps: float = 1e-6, norm=True, interleaved=False, positions=None, q_out=None,
                     max_kv_len=None, ws=None, stream=None):
    """Norm and rotation of q [T, h_q, d] and k [T, h_kv, d]; k and v go to the paged caches
    [n_pages, page_size, h_kv, d] at the places that kv_len (the new tokens counted) gives them.

    ``cos_sin`` [positions, rot_dim] fp32: cosines, then sines (None or no columns: no rotation).
    ``positions`` [T] int32: rotate by these instead of the places.  ``q_out`` may be q.  Returns q_out.
    """
    if _elsewhere(q, stream):
        with _context(q, stream):
            return gdn_qk_norm_rope(q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len,
                                    q_weight=q_weight, k_weight=k_weight, eps=eps, norm=norm, interleaved=interleaved,
                                    positions=positions, q_out=q_out, max_kv_len=max_kv_len, ws=ws)
    lib, w = load(), "gdn_qk_norm_rope"
    n = _paged_lists(w, block_table, cu_seqlens, kv_len)
    d = _paged(w, q, k_cache, v_cache, block_table, n, max_kv_len)
    (T, h, dim), hk, e = q.shape, d.h_kv, q.dtype
    d.q_stride = _rows(q, (T, h, dim), e, w + ": q")
    d.k_stride = _rows(k, (T, hk, dim), e, w + ": k")
    d.v_stride = _rows(v, (T, hk, dim), e, w + ": v")
    _whole(q_weight, (dim,), _f32, w + ": q_weight", True)
    _whole(k_weight, (dim,), _f32, w + ": k_weight", True)
    if cos_sin is not None:
        _need(cos_sin.dim() == 2, GDN_ERR_SHAPE, w + ": cos_sin [positions, rot_dim]")
        d.max_pos, d.rot_dim = cos_sin.shape
        _whole(cos_sin, tuple(cos_sin.shape), _f32, w + ": cos_sin")
    _whole(positions, (T,), _i32, w + ": positions", True)
    if q_out is None:
        q_out = torch.empty((T, h, dim), dtype=e, device=q.device)
    d.o_stride = _rows(q_out, (T, h, dim), e, w + ": q_out")
    d.interleaved, d.norm, d.eps = int(bool(interleaved)), int(bool(norm)), float(eps)
    dev = _device(w, q, k, v, q_weight, k_weight, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len,
                  positions, q_out)
    ws = _workspace(ws, 256, dev, w)
    _check(lib.gdn_qk_norm_rope(_byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(q_weight), _p(k_weight),
                                _p(cos_sin), block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(),
                                _p(positions), k_cache.data_ptr(), v_cache.data_ptr(), q_out.data_ptr(),
                                ws.data_ptr(), ws.numel(), _current(dev)), w)
    return q_out


def gdn_paged_attn(q, k_cache, v_cache, block_table, cu_seqlens, kv_len, *, max_kv_len=None, scale=None, o=None,
                   lse=None, ws=None, stream=None):
    """Attention of new tokens q [T, h_q, d] over the paged caches, each to its position and before.

    ``max_kv_len``: no kv_len is larger (None: all that the block table holds; a tight bound spreads
    the work better).  ``scale``: of the scores (None: d ** -0.5).  ``lse``: a tensor [T, h_q] fp32 or
    True (allocate).  ``ws``, when given, holds gdn_paged_workspace_bytes(make_paged_desc(...)) bytes.
    Returns o, or (o, lse) where lse was asked for.
    """
    if _elsewhere(q, stream):
        with _context(q, stream):
            return gdn_paged_attn(q, k_cache, v_cache, block_table, cu_seqlens, kv_len, max_kv_len=max_kv_len,
                                  scale=scale, o=o, lse=lse, ws=ws)
    lib, w = load(), "gdn_paged_attn"
    n = _paged_lists(w, block_table, cu_seqlens, kv_len)
    d = _paged(w, q, k_cache, v_cache, block_table, n, max_kv_len)
    T, h, dim = q.shape
    d.q_stride = _rows(q, (T, h, dim), q.dtype, w + ": q")
    if o is None:
        o = torch.empty((T, h, dim), dtype=q.dtype, device=q.device)
    d.o_stride = _rows(o, (T, h, dim), q.dtype, w + ": o")
    if lse is True:
        lse = torch.empty((T, h), dtype=_f32, device=q.device)
    elif lse is False:
        lse = None
    _whole(lse, (T, h), _f32, w + ": lse", True)
    if scale is not None:
        d.scale = float(scale)
    dev = _device(w, q, k_cache, v_cache, block_table, cu_seqlens, kv_len, o, lse)
    if ws is None:
        ws = _workspace(None, max(256, gdn_paged_workspace_bytes(d)), dev, w)
    else:
        _workspace(ws, 0, dev, w)
    _check(lib.gdn_paged_attn(_byref(d), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                              block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(), o.data_ptr(), _p(lse),
                              ws.data_ptr(), ws.numel(), _current(dev)), w)
    return o if lse is None else (o, lse)
