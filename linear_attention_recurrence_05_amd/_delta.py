"""ctypes marshalling of the delta-rule, gated-norm and block-norm entry points of
libkda (see ``include/kda.h`` for the contract).

Like ``_linear``: the functions named ``kda_*`` take torch tensors in the layouts
``kda.h`` documents and pass their device pointers through; the others also
allocate what the caller does not give.  Every tensor must be contiguous, on
one CUDA device, and of the exact shape.  ``stream`` (None: the current stream
of the tensors' device) is where the call runs; allocating helpers allocate on
it, so their results belong to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import _i, _vp, lib
from ._linear import _F32, _I32, _Call, _code, _dims, _empty, _f, _on, _pool, _z

KDA_GATE_SIGMOID = 0
KDA_GATE_SILU = 1
KDA_MAX_NORM_WIDTH = 16384
_GATES = {"sigmoid": KDA_GATE_SIGMOID, "silu": KDA_GATE_SILU}

_ll = ctypes.c_longlong
_lib._SIGNATURES.update({
    "kda_delta_prefill_workspace_bytes": ([_i] * 7, _z),
    "kda_delta_prefill": ([_vp] * 5 + [_f] + [_vp] * 4 + [_i] * 7 + [_vp, _z, _vp], _i),
    "kda_delta_prefill_paged": ([_vp] * 5 + [_f, _vp, _i] + [_vp] * 4 + [_i] * 7 + [_vp, _z, _vp], _i),
    "kda_delta_backward_workspace_bytes": ([_i] * 7, _z),
    "kda_delta_backward": ([_vp] * 5 + [_f] + [_vp] * 10 + [_i] * 7 + [_vp, _z, _vp], _i),
    "kda_delta_decode_step": ([_vp] * 5 + [_f] + [_vp] * 2 + [_i] * 6 + [_vp], _i),
    "kda_delta_decode_step_paged": ([_vp] * 5 + [_f, _vp, _i] + [_vp] * 2 + [_i] * 6 + [_vp], _i),
    "kda_gated_norm": ([_vp] * 3 + [_i, _f, _vp, _ll, _i, _i, _vp], _i),
    "kda_gated_norm_backward_workspace_bytes": ([_ll, _i, _i], _z),
    "kda_gated_norm_backward": ([_vp] * 3 + [_i, _f] + [_vp] * 4 + [_ll, _i, _i, _vp, _z, _vp], _i),
    "kda_block_norm": ([_vp] * 5 + [_i, _f, _f] + [_vp] * 2 + [_ll, _i, _i, _vp], _i),
    "kda_block_norm_backward_workspace_bytes": ([_ll, _i, _i], _z),
    "kda_block_norm_backward": ([_vp] * 5 + [_i, _f, _f] + [_vp] * 7 + [_ll, _i, _i, _vp, _z, _vp], _i),
})


# ----------------------------------------------------------------- gated delta rule

def kda_delta_prefill_workspace_bytes(B, T, H, H_k, d_k, d_v, dtype) -> int:
    return int(lib().kda_delta_prefill_workspace_bytes(B, T, H, H_k, d_k, d_v, _code(dtype)))


def kda_delta_backward_workspace_bytes(B, T, H, H_k, d_k, d_v, dtype) -> int:
    return int(lib().kda_delta_backward_workspace_bytes(B, T, H, H_k, d_k, d_v, _code(dtype)))


def kda_delta_prefill(q, k, v, g, beta, scale, S0, o, S_T, lens=None, workspace=None, stream=None):
    """C entry point kda_delta_prefill."""
    c = _Call("kda_delta_prefill", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_delta_prefill", stream, c("q", q, (B, T, Hk, dk)), c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (B, T, H), _F32), c("beta", beta, (B, T, H), _F32),
          float(scale), c("S0", S0, (B, H, dk, dv), _F32, True), c("lens", lens, (B,), _I32, True),
          c("o", o, (B, T, H, dv)), c("S_T", S_T, (B, H, dk, dv), _F32, True),
          B, T, H, Hk, dk, dv, c.code, ws, nbytes)


def kda_delta_prefill_paged(q, k, v, g, beta, scale, pool, slots_in, slots_out, o, lens=None,
                            workspace=None, stream=None):
    """C entry point kda_delta_prefill_paged: states from pool[slots_in[b]] into
    pool[slots_out[b]] (either table may be None)."""
    c = _Call("kda_delta_prefill_paged", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_delta_prefill_paged", stream, c("q", q, (B, T, Hk, dk)), c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (B, T, H), _F32), c("beta", beta, (B, T, H), _F32),
          float(scale), pp, n_slots, c("slots_in", slots_in, (B,), _I32, True),
          c("slots_out", slots_out, (B,), _I32, True), c("lens", lens, (B,), _I32, True),
          c("o", o, (B, T, H, dv)), B, T, H, Hk, dk, dv, c.code, ws, nbytes)


def delta_prefill(q, k, v, g, beta, scale=1.0, S0=None, lens=None, want_state=True, o=None,
                  stream=None):
    """kda_delta_prefill with S_T, the workspace and (unless given) o allocated;
    an allocated o is zero past the lengths.  Returns (o, S_T or None)."""
    c = _Call("delta_prefill", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    with _on(q, stream):
        if o is None:
            new = torch.empty if lens is None else torch.zeros
            o = new((B, T, H, dv), dtype=q.dtype, device=q.device)
        S_T = torch.empty((B, H, dk, dv), dtype=_F32, device=q.device) if want_state else None
        ws = _empty(lib().kda_delta_prefill_workspace_bytes(B, T, H, Hk, dk, dv, c.code), q.device)
        kda_delta_prefill(q, k, v, g, beta, scale, S0, o, S_T, lens, ws, stream)
    return o, S_T


def kda_delta_backward(q, k, v, g, beta, scale, S0, dO, dS_T, dq, dk, dv, dg, dbeta, dS0, lens=None,
                       workspace=None, stream=None):
    """C entry point kda_delta_backward."""
    c = _Call("kda_delta_backward", q, 4)
    B, T, H, dvv, Hk, dkk = _dims(c, q, v, 4)
    qk, vo, st, gt = (B, T, Hk, dkk), (B, T, H, dvv), (B, H, dkk, dvv), (B, T, H)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_delta_backward", stream, c("q", q, qk), c("k", k, qk), c("v", v, vo),
          c("g", g, gt, _F32), c("beta", beta, gt, _F32), float(scale), c("S0", S0, st, _F32, True),
          c("lens", lens, (B,), _I32, True), c("dO", dO, vo), c("dS_T", dS_T, st, _F32, True),
          c("dq", dq, qk), c("dk", dk, qk), c("dv", dv, vo), c("dg", dg, gt, _F32),
          c("dbeta", dbeta, gt, _F32), c("dS0", dS0, st, _F32, True), B, T, H, Hk, dkk, dvv, c.code,
          ws, nbytes)


def delta_backward(q, k, v, g, beta, dO, scale=1.0, S0=None, dS_T=None, lens=None, want_dS0=True,
                   dq=None, dk=None, dv=None, dg=None, dbeta=None, stream=None):
    """kda_delta_backward with the workspace and the gradients that are not given
    allocated; allocated ones are zero past the lengths.  Returns a dict with
    dq, dk, dv, dg, dbeta, dS0."""
    c = _Call("delta_backward", q, 4)
    B, T, H, dvv, Hk, dkk = _dims(c, q, v, 4)
    with _on(q, stream):
        new = torch.empty if lens is None else torch.zeros
        dq, dk, dv, dg, dbeta = (new(s, dtype=t, device=q.device) if d is None else d for s, t, d in
                                 (((B, T, Hk, dkk), q.dtype, dq), ((B, T, Hk, dkk), q.dtype, dk),
                                  ((B, T, H, dvv), q.dtype, dv), ((B, T, H), _F32, dg), ((B, T, H), _F32, dbeta)))
        dS0 = torch.empty((B, H, dkk, dvv), dtype=_F32, device=q.device) if want_dS0 else None
        ws = _empty(lib().kda_delta_backward_workspace_bytes(B, T, H, Hk, dkk, dvv, c.code), q.device)
        kda_delta_backward(q, k, v, g, beta, scale, S0, dO, dS_T, dq, dk, dv, dg, dbeta, dS0, lens,
                           ws, stream)
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dS0=dS0)


def kda_delta_decode_step(q, k, v, g, beta, scale, S, o, stream=None):
    """C entry point kda_delta_decode_step; S is updated in place."""
    c = _Call("kda_delta_decode_step", q, 3)
    B, H, dv, Hk, dk = _dims(c, q, v, 3)
    c.run("kda_delta_decode_step", stream, c("q", q, (B, Hk, dk)), c("k", k, (B, Hk, dk)),
          c("v", v, (B, H, dv)), c("g", g, (B, H), _F32), c("beta", beta, (B, H), _F32), float(scale),
          c("S", S, (B, H, dk, dv), _F32), c("o", o, (B, H, dv)), B, H, Hk, dk, dv, c.code)


def kda_delta_decode_step_paged(q, k, v, g, beta, scale, pool, slots, o, stream=None):
    """C entry point kda_delta_decode_step_paged: pool[slots[b]] updated in place."""
    c = _Call("kda_delta_decode_step_paged", q, 3)
    B, H, dv, Hk, dk = _dims(c, q, v, 3)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    c.run("kda_delta_decode_step_paged", stream, c("q", q, (B, Hk, dk)), c("k", k, (B, Hk, dk)),
          c("v", v, (B, H, dv)), c("g", g, (B, H), _F32), c("beta", beta, (B, H), _F32), float(scale),
          pp, n_slots, c("slots", slots, (B,), _I32), c("o", o, (B, H, dv)), B, H, Hk, dk, dv, c.code)


def delta_decode_step(q, k, v, g, beta, S, scale=1.0, stream=None):
    """kda_delta_decode_step with o allocated (S updated in place).  Returns o."""
    with _on(v, stream):
        o = torch.empty_like(v)
        kda_delta_decode_step(q, k, v, g, beta, scale, S, o, stream)
    return o


# ----------------------------------------------------------------- norms

def _rows_call(where, x):
    """The call's checks and its rows: x [..., d] as rows of d elements."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{where}: expected a torch.Tensor, got {type(x).__name__}")
    if x.dim() < 1:
        raise ValueError(f"{where}: expected at least one dimension")
    c = _Call(where, x, x.dim())
    d = x.shape[-1]
    return c, tuple(x.shape), (x.numel() // d if d else 0), d


def _gate(c, act):
    if act not in _GATES:
        raise ValueError(f"{c.where}: act must be one of {sorted(_GATES)}, got {act!r}")
    return _GATES[act]


def kda_gated_norm(x, z, w, act, eps, y, stream=None):
    """C entry point kda_gated_norm: rows x, z, y [..., d], w fp32 [d] or None, act
    "sigmoid" or "silu"; y may be x."""
    c, s, rows, d = _rows_call("kda_gated_norm", x)
    c.run("kda_gated_norm", stream, c("x", x, s), c("z", z, s), c("w", w, (d,), _F32, True),
          _gate(c, act), float(eps), c("y", y, s), rows, d, c.code)


def gated_norm(x, z, w=None, act="silu", eps=1e-6, stream=None):
    """kda_gated_norm with y allocated.  Returns y."""
    with _on(x, stream):
        y = torch.empty_like(x)
        kda_gated_norm(x, z, w, act, eps, y, stream)
    return y


def kda_gated_norm_backward_workspace_bytes(rows, d, dtype) -> int:
    return int(lib().kda_gated_norm_backward_workspace_bytes(rows, d, _code(dtype)))


def kda_gated_norm_backward(x, z, w, act, eps, dy, dx, dz, dw, workspace=None, stream=None):
    """C entry point kda_gated_norm_backward; dw may be None, dx may be dy."""
    c, s, rows, d = _rows_call("kda_gated_norm_backward", x)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_gated_norm_backward", stream, c("x", x, s), c("z", z, s), c("w", w, (d,), _F32, True),
          _gate(c, act), float(eps), c("dy", dy, s), c("dx", dx, s), c("dz", dz, s),
          c("dw", dw, (d,), _F32, True), rows, d, c.code, ws, nbytes)


def gated_norm_backward(x, z, w, dy, act="silu", eps=1e-6, stream=None):
    """kda_gated_norm_backward with the gradients and the workspace allocated.
    Returns a dict with dx, dz, dw (None without w)."""
    c, _, rows, d = _rows_call("gated_norm_backward", x)
    with _on(x, stream):
        dx, dz = torch.empty_like(x), torch.empty_like(x)
        dw = ws = None
        if w is not None:
            dw = torch.empty(d, dtype=_F32, device=x.device)
            ws = _empty(lib().kda_gated_norm_backward_workspace_bytes(rows, d, c.code), x.device)
        kda_gated_norm_backward(x, z, w, act, eps, dy, dx, dz, dw, ws, stream)
    return dict(dx=dx, dz=dz, dw=dw)


def kda_block_norm(y, z, w_y, r, w_n, norm_y, scale, eps, h, n, stream=None):
    """C entry point kda_block_norm: rows y, z, r, h, n [..., D]; z, w_y and w_n may be
    None, and without y all that belongs to it (z, w_y, h) is None.  h may be r, and n
    may be y (without y: r)."""
    c, s, rows, D = _rows_call("kda_block_norm", r)
    c.run("kda_block_norm", stream, c("y", y, s, None, True), c("z", z, s, None, True),
          c("w_y", w_y, (D,), _F32, True), c("r", r, s), c("w_n", w_n, (D,), _F32, True),
          int(bool(norm_y)), float(scale), float(eps), c("h", h, s, None, y is None), c("n", n, s),
          rows, D, c.code)


def block_norm(y, r, z=None, w_y=None, w_n=None, norm_y=False, scale=1.0, eps=1e-6, stream=None):
    """kda_block_norm with h and n allocated.  Returns (h, n); without y, h is r itself."""
    with _on(r, stream):
        h, n = None if y is None else torch.empty_like(r), torch.empty_like(r)
        kda_block_norm(y, z, w_y, r, w_n, norm_y, scale, eps, h, n, stream)
    return (r if y is None else h), n


def kda_block_norm_backward_workspace_bytes(rows, D, dtype) -> int:
    return int(lib().kda_block_norm_backward_workspace_bytes(rows, D, _code(dtype)))


def kda_block_norm_backward(y, z, w_y, h, w_n, norm_y, scale, eps, dn, dh, dr, dy, dz, dw_y, dw_n,
                            workspace=None, stream=None):
    """C entry point kda_block_norm_backward; dh, dw_y and dw_n may be None, and without y
    (or z) its gradients are None too.  dr may be dh."""
    c, s, rows, D = _rows_call("kda_block_norm_backward", h)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_block_norm_backward", stream, c("y", y, s, None, True), c("z", z, s, None, True),
          c("w_y", w_y, (D,), _F32, True), c("h", h, s), c("w_n", w_n, (D,), _F32, True),
          int(bool(norm_y)), float(scale), float(eps), c("dn", dn, s), c("dh", dh, s, None, True),
          c("dr", dr, s), c("dy", dy, s, None, y is None), c("dz", dz, s, None, z is None),
          c("dw_y", dw_y, (D,), _F32, True), c("dw_n", dw_n, (D,), _F32, True), rows, D, c.code,
          ws, nbytes)


def block_norm_backward(y, h, dn, dh=None, z=None, w_y=None, w_n=None, norm_y=False, scale=1.0,
                        eps=1e-6, stream=None):
    """kda_block_norm_backward with the gradients and the workspace allocated.  Returns a
    dict with dr, dy, dz, dw_y, dw_n (None where the input is)."""
    c, _, rows, D = _rows_call("block_norm_backward", h)
    with _on(h, stream):
        dr = torch.empty_like(h)
        dy, dz = (None if t is None else torch.empty_like(h) for t in (y, z))
        dw_y, dw_n = (None if t is None else torch.empty(D, dtype=_F32, device=h.device) for t in (w_y, w_n))
        ws = None
        if dw_y is not None or dw_n is not None:
            ws = _empty(lib().kda_block_norm_backward_workspace_bytes(rows, D, c.code), h.device)
        kda_block_norm_backward(y, z, w_y, h, w_n, norm_y, scale, eps, dn, dh, dr, dy, dz, dw_y,
                                dw_n, ws, stream)
    return dict(dr=dr, dy=dy, dz=dz, dw_y=dw_y, dw_n=dw_n)
