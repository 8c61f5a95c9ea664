"""Python binding of the suffix and decode operators (see include/gdn.h).

As the rest of the package: the functions carry the names of the C entry points and marshal
arguments.  Checks of dtypes, shapes, strides and devices, output allocation and the call itself are
in the native module (csrc/gdn_torch.cpp): a refusal raises GdnError with the matching status before
anything is enqueued.  ``ws`` is a zero-filled uint8 workspace that the caller keeps (one for each
stream or graph that may run at the same time); a call without it makes a new one.  Calls run on
torch's current stream of the tensors' device, or on ``stream``.  As everywhere in this package, autograd is
not involved: outputs carry no gradient, whatever the inputs require, and what is updated in place (states,
caches, given outputs) is so without a new version of the tensor.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from ._lib import (GDN_BF16, GDN_ERR_DTYPE, GDN_ERR_SHAPE, GDN_F32, GdnError, GdnPagedDesc, GdnSsmDesc, load)

_DT = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_gdn_torch.so")
_native = None


def _load():
    """The native module, given the library's entry points; raises if either is not built."""
    global _native
    if _native is None:
        lib = load()
        if not os.path.exists(BINDING_PATH):
            raise ImportError("_gdn_torch.so is not built: run `python -m gated_deltanet_state_gdn_amd.build`"
                              " (or __graft_entry__.build())")
        spec = importlib.util.spec_from_file_location("_gdn_torch", BINDING_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.bind(GdnError, _raw_stream,
               *(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
                   "gdn_conv", "gdn_conv_step", "gdn_ssm_scan", "gdn_ssm_step", "gdn_step", "gdn_qk_norm_rope",
                   "gdn_paged_attn", "gdn_ssm_workspace_bytes", "gdn_paged_workspace_bytes")))
        _native = m
    return _native


# the current stream's handle, without a Stream object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(stream, x):
    # allocations and the workspace's fill belong to the stream of the call
    if x.device != stream.device:
        raise GdnError(GDN_ERR_SHAPE, "the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _silu(activation):
    if activation not in ("silu", None):
        raise GdnError(GDN_ERR_SHAPE, "activation: 'silu' or None")
    return activation is not None


def gdn_conv(x, weight, cu_seqlens, *, bias=None, state0=None, state_out=True, activation="silu", y=None,
             ws=None, stream=None):
    """Short causal convolution of packed prompts: x [T, channels], weight [channels, width] fp32.

    ``state0`` [n_seqs, width - 1, channels]: the inputs in front of each sequence (None: zero);
    ``state_out``: a tensor (may be state0), True (allocate) or None.  Returns (y, state_out or None).
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_conv(x, weight, cu_seqlens, bias=bias, state0=state0, state_out=state_out,
                            activation=activation, y=y, ws=ws)
    return (_native or _load()).conv(x, weight, cu_seqlens, bias, state0, state_out, _silu(activation), y, ws)


def gdn_conv_step(x, weight, state, *, slots=None, bias=None, activation="silu", y=None, ws=None, stream=None):
    """One token per row: x [rows, channels]; ``state`` [n_slots, width - 1, channels] is updated in
    place.  ``slots`` [rows] int32: the state of each row, -1 for a padded one (None: state i for row
    i).  Returns y."""
    if stream is not None:
        with _on(stream, x):
            return gdn_conv_step(x, weight, state, slots=slots, bias=bias, activation=activation, y=y, ws=ws)
    return (_native or _load()).conv_step(x, weight, state, slots, bias, _silu(activation), y, ws)


def _code(x):
    dt = _DT.get(x.dtype)
    if dt is None:
        raise GdnError(GDN_ERR_DTYPE, "float32 or bfloat16 wanted")
    return dt


def make_ssm_desc(x, B, n_seqs, *, total_out_tokens=None, n_slots=0, softplus=True) -> GdnSsmDesc:
    """Sizes of a state space call (x [T, h_v, d_v], B [T, h_qk, d_k]), for its workspace."""
    if x.dim() != 3 or B.dim() != 3:
        raise GdnError(GDN_ERR_SHAPE, "make_ssm_desc: x [T, h_v, d_v], B [T, h_qk, d_k]")
    T, h, p = x.shape
    g, k = B.shape[1:]
    return GdnSsmDesc(int(n_seqs), int(n_slots), g, h, k, p, _code(x), int(bool(softplus)), T,
                      T if total_out_tokens is None else int(total_out_tokens), h * p, g * k, g * k, h, h * p)


def gdn_ssm_workspace_bytes(desc: GdnSsmDesc) -> int:
    return int(load().gdn_ssm_workspace_bytes(ctypes.byref(desc)))


def gdn_ssm_scan(x, B, C, dt, A, cu_seqlens, *, D=None, dt_bias=None, softplus=True, r=None, total_out_tokens=None,
                 S0=None, S_out=None, y_out=True, cu_out=None, ws=None, stream=None):
    """Selective state space scan of packed prompts: x [T, h_v, d_v], B, C [T, h_qk, d_k], dt [T, h_v].

    ``r`` [n_seqs] int32: only the last r[n] tokens of each sequence (then ``total_out_tokens`` = their
    sum, y packed per window, ``cu_out`` as for gdn_replay).  ``S0`` [n_seqs, h_v, d_k, d_v]: the states
    to start from; ``S_out`` may be S0.  ``y_out``: a tensor, True (allocate) or None.  ``ws``, when
    given, holds gdn_ssm_workspace_bytes(make_ssm_desc(...)) bytes.  Returns (S_out, y or None, cu_out).
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_ssm_scan(x, B, C, dt, A, cu_seqlens, D=D, dt_bias=dt_bias, softplus=softplus, r=r,
                                total_out_tokens=total_out_tokens, S0=S0, S_out=S_out, y_out=y_out, cu_out=cu_out,
                                ws=ws)
    return (_native or _load()).scan(x, B, C, dt, A, cu_seqlens, D, dt_bias, softplus, r, total_out_tokens, S0, S_out,
                                     y_out, cu_out, ws)


def gdn_ssm_step(x, B, C, dt, A, S, *, slots=None, D=None, dt_bias=None, softplus=True, y=None, ws=None, stream=None):
    """One token per row of the state space recurrence; ``S`` [n_slots, h_v, d_k, d_v] is updated in
    place, ``slots`` as for gdn_conv_step.  Returns y [rows, h_v, d_v]."""
    if stream is not None:
        with _on(stream, x):
            return gdn_ssm_step(x, B, C, dt, A, S, slots=slots, D=D, dt_bias=dt_bias, softplus=softplus, y=y, ws=ws)
    return (_native or _load()).ssm_step(x, B, C, dt, A, S, slots, D, dt_bias, softplus, y, ws)


def gdn_step(q, k, v, g, beta, S, *, slots=None, o=None, scale: float = 1.0, o_dtype=None, ws=None, stream=None):
    """One token per row of the gated delta rule: q, k [rows, h_qk, d_k], v [rows, h_v, d_v], g, beta
    [rows, h_v] fp32; ``S`` [n_slots, h_v, d_k, d_v] is updated in place, ``slots`` as for
    gdn_conv_step.  Returns o [rows, h_v, d_v]."""
    if stream is not None:
        with _on(stream, q):
            return gdn_step(q, k, v, g, beta, S, slots=slots, o=o, scale=scale, o_dtype=o_dtype, ws=ws)
    return (_native or _load()).step(q, k, v, g, beta, S, slots, o, scale, _f32_out(q, o_dtype), ws)


def _f32_out(q, o_dtype):
    if o_dtype is None or o_dtype is q.dtype:
        return False
    if o_dtype is not torch.float32:
        raise GdnError(GDN_ERR_DTYPE, "gdn_step: o has q's dtype or float32")
    return True


def make_paged_desc(q, k_cache, block_table, n_seqs, *, max_kv_len=None) -> GdnPagedDesc:
    """Sizes of a paged call (q [T, h_q, d], caches [n_pages, page_size, h_kv, d]), for
    gdn_paged_attn's workspace.  ``max_kv_len``: the largest kv_len that will be passed (None: all
    that the block table holds)."""
    if q.dim() != 3 or k_cache.dim() != 4 or block_table.dim() != 2:
        raise GdnError(GDN_ERR_SHAPE, "make_paged_desc: q [T, h_q, d], caches [n_pages, page_size, h_kv, d],"
                                      " block_table [n_seqs, max_pages]")
    (T, h, d), (pages, ps, hk, _) = q.shape, k_cache.shape
    hold = min(block_table.shape[1] * ps, 1 << 30)
    return GdnPagedDesc(n_seqs=int(n_seqs), h_q=h, h_kv=hk, d=d, dtype=_code(q), page_size=ps, n_pages=pages,
                        max_pages=block_table.shape[1], max_kv_len=hold if max_kv_len is None else min(int(max_kv_len), hold),
                        scale=d ** -0.5, total_tokens=T, q_stride=h * d, k_stride=hk * d, v_stride=hk * d,
                        o_stride=h * d, page_stride=ps * hk * d, token_stride=hk * d, head_stride=d)


def gdn_paged_workspace_bytes(desc: GdnPagedDesc) -> int:
    return int(load().gdn_paged_workspace_bytes(ctypes.byref(desc)))


def gdn_qk_norm_rope(q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len, *, q_weight=None,
                     k_weight=None, eps: float = 1e-6, norm=True, interleaved=False, positions=None, q_out=None,
                     max_kv_len=None, ws=None, stream=None):
    """Norm and rotation of q [T, h_q, d] and k [T, h_kv, d]; k and v go to the paged caches
    [n_pages, page_size, h_kv, d] at the places that kv_len (the new tokens counted) gives them.

    ``cos_sin`` [positions, rot_dim] fp32: cosines, then sines (None or no columns: no rotation).
    ``positions`` [T] int32: rotate by these instead of the places.  ``q_out`` may be q.  Returns q_out.
    """
    if stream is not None:
        with _on(stream, q):
            return gdn_qk_norm_rope(q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len,
                                    q_weight=q_weight, k_weight=k_weight, eps=eps, norm=norm, interleaved=interleaved,
                                    positions=positions, q_out=q_out, max_kv_len=max_kv_len, ws=ws)
    return (_native or _load()).rope(q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_len, q_weight,
                                     k_weight, eps, norm, interleaved, positions, q_out, max_kv_len, ws)


def gdn_paged_attn(q, k_cache, v_cache, block_table, cu_seqlens, kv_len, *, max_kv_len=None, scale=None, o=None,
                   lse=None, ws=None, stream=None):
    """Attention of new tokens q [T, h_q, d] over the paged caches, each to its position and before.

    ``max_kv_len``: no kv_len is larger (None: all that the block table holds; a tight bound spreads
    the work better).  ``scale``: of the scores (None: d ** -0.5).  ``lse``: a tensor [T, h_q] fp32 or
    True (allocate).  ``ws``, when given, holds gdn_paged_workspace_bytes(make_paged_desc(...)) bytes.
    Returns o, or (o, lse) where lse was asked for.
    """
    if stream is not None:
        with _on(stream, q):
            return gdn_paged_attn(q, k_cache, v_cache, block_table, cu_seqlens, kv_len, max_kv_len=max_kv_len,
                                  scale=scale, o=o, lse=lse, ws=ws)
    return (_native or _load()).attn(q, k_cache, v_cache, block_table, cu_seqlens, kv_len, max_kv_len, scale, o, lse,
                                     ws)
