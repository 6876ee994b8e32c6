"""ctypes marshalling of the linear-attention, draft-tree and norm entry points
of libkda (see ``include/kda.h`` for the contract).

Like ``_lib``: the functions named ``kda_*`` take torch tensors in the layouts
``kda.h`` documents and pass their device pointers through; the others also
allocate what the caller does not give.  Every tensor must be contiguous, on
one CUDA device, and of the exact shape.  ``stream`` (None: the current stream
of the tensors' device) is where the call runs; allocating helpers allocate on
it, so their results belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import KDA_BF16, KDA_F32, _check, _i, _vp, lib

KDA_MAX_TREE_TOKENS = 64
KDA_NORM_L2 = 0
KDA_NORM_RMS = 1
_NORMS = {"l2": KDA_NORM_L2, "rms": KDA_NORM_RMS}

_f, _z = ctypes.c_float, ctypes.c_size_t
_lib._SIGNATURES.update({
    "kda_linear_prefill_workspace_bytes": ([_i] * 7, _z),
    "kda_linear_prefill": ([_vp] * 4 + [_f] + [_vp] * 4 + [_i] * 7 + [_vp, _z, _vp], _i),
    "kda_linear_prefill_paged": ([_vp] * 4 + [_f, _vp, _i] + [_vp] * 4 + [_i] * 7
                                 + [_vp, _z, _vp], _i),
    "kda_linear_backward_workspace_bytes": ([_i] * 7, _z),
    "kda_linear_backward": ([_vp] * 4 + [_f] + [_vp] * 8 + [_i] * 7 + [_vp, _z, _vp], _i),
    "kda_linear_decode_step": ([_vp] * 4 + [_f] + [_vp] * 2 + [_i] * 6 + [_vp], _i),
    "kda_linear_decode_step_paged": ([_vp] * 4 + [_f, _vp, _i] + [_vp] * 2 + [_i] * 6 + [_vp], _i),
    "kda_linear_tree": ([_vp] * 4 + [_f] + [_vp] * 3 + [_i] * 7 + [_vp], _i),
    "kda_linear_tree_paged": ([_vp] * 4 + [_f, _vp, _i] + [_vp] * 3 + [_i] * 7 + [_vp], _i),
    "kda_linear_tree_commit": ([_vp] * 7 + [_i] * 7 + [_vp], _i),
    "kda_linear_tree_commit_paged": ([_vp] * 6 + [_i] + [_vp] * 2 + [_i] * 7 + [_vp], _i),
    "kda_qk_norm_rope": ([_vp] * 6 + [_i, _f, _i, _i] + [_vp] * 2 + [_i] * 6 + [_vp], _i),
    "kda_qk_norm_rope_backward_workspace_bytes": ([_i] * 6, _z),
    "kda_qk_norm_rope_backward": ([_vp] * 6 + [_i, _f, _i, _i] + [_vp] * 6 + [_i] * 6
                                  + [_vp, _z, _vp], _i),
})

_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)

_F32 = torch.float32
_I32 = torch.int32
_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}


def _refuse(where, name, t, dev, dtype, shape):
    if t is None:
        raise ValueError(f"{where}: {name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{where}: {name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{where}: {name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{where}: {name} must be contiguous")


class _Call:
    """The checks of one call's tensors against the first one's device and type."""

    __slots__ = ("where", "index", "dt", "code")

    @property
    def dev(self):
        return torch.device("cuda", self.index) if self.index >= 0 else torch.device("cpu")

    def __init__(self, where, ref, ndim):
        self.where = where
        if not isinstance(ref, torch.Tensor):
            raise TypeError(f"{where}: expected a torch.Tensor, got {type(ref).__name__}")
        self.index, self.dt = ref.get_device(), ref.dtype      # index -1: host memory
        if not ref.is_cuda and _lib._DEVICE_TYPE == "cuda":
            raise ValueError(f"{where}: tensors must be on a CUDA device, got {ref.device}")
        code = _CODES.get(self.dt)
        if code is None:
            raise ValueError(f"{where}: q, k, v and o must be bfloat16 or float32, got {self.dt}")
        if ref.dim() != ndim:
            raise ValueError(f"{where}: expected {ndim} dimensions, got shape {tuple(ref.shape)}")
        self.code = code

    def __call__(self, name, t, shape, dtype=None, optional=False):
        """The tensor's address, after its checks."""
        if t is None and optional:
            return None
        if dtype is None:
            dtype = self.dt
        try:
            if (t.dtype is dtype and t.shape == shape and t.get_device() == self.index
                    and t.is_contiguous()):
                return t.data_ptr()
        except AttributeError:
            pass
        _refuse(self.where, name, t, self.dev, dtype, shape)

    def workspace(self, ws):
        """(address, bytes); any dtype, the library checks the size."""
        if ws is None:
            return None, 0
        if not isinstance(ws, torch.Tensor) or ws.device != self.dev or not ws.is_contiguous():
            raise ValueError(f"{self.where}: workspace must be a contiguous tensor on {self.dev}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def run(self, name, stream, *args):
        """Calls the entry point on `stream`, with the tensors' device current."""
        i = self.index
        if i < 0:
            raise ValueError(f"{self.where}: tensors must be on a CUDA device, got {self.dev}")
        # torch's own bindings for the current stream and device: the public
        # functions around them cost several times what they do
        raw = _current_stream(i) if stream is None else _raw(stream)
        if i == _current_device():
            st = _entry(name)(*args, raw)
        else:
            with torch.cuda.device(self.dev):
                st = _entry(name)(*args, raw)
        if st:
            _check(st, name)


_entries = {}


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(lib(), name)
    return fn


def _raw(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_NO_STREAM = contextlib.nullcontext()


def _on(t, stream):
    """Allocations inside belong to the stream that the call runs on."""
    if stream is None or not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        return _NO_STREAM
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    return torch.cuda.stream(stream)


def _code(dtype):
    return dtype if isinstance(dtype, int) else (KDA_BF16 if dtype == torch.bfloat16 else KDA_F32)


def _dims(c, q, v, ndim):
    """(lead sizes.., H, d_v, H_k, d_k) from q [.., H_k, d_k] and v [.., H, d_v]."""
    if not isinstance(v, torch.Tensor) or v.dim() != ndim:
        raise ValueError(f"{c.where}: v must be a tensor with {ndim} dimensions")
    if ndim == 3:
        B, Hk, dk = q.shape
        _, H, dv = v.shape
        return B, H, dv, Hk, dk
    B, T, Hk, dk = q.shape
    _, _, H, dv = v.shape
    return B, T, H, dv, Hk, dk


def _pool(c, pool, H, dk, dv):
    if not isinstance(pool, torch.Tensor) or pool.dim() != 4:
        raise ValueError(f"{c.where}: pool must be a tensor [n_slots, H, d_k, d_v]")
    return c("pool", pool, (pool.shape[0], H, dk, dv), _F32), pool.shape[0]


def _empty(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# ----------------------------------------------------------------- linear attention

def kda_linear_prefill_workspace_bytes(B, T, H, H_k, d_k, d_v, dtype) -> int:
    return int(lib().kda_linear_prefill_workspace_bytes(B, T, H, H_k, d_k, d_v, _code(dtype)))


def kda_linear_backward_workspace_bytes(B, T, H, H_k, d_k, d_v, dtype) -> int:
    return int(lib().kda_linear_backward_workspace_bytes(B, T, H, H_k, d_k, d_v, _code(dtype)))


def kda_linear_prefill(q, k, v, g, scale, S0, o, S_T, lens=None, workspace=None, stream=None):
    """C entry point kda_linear_prefill."""
    c = _Call("kda_linear_prefill", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_linear_prefill", stream, c("q", q, (B, T, Hk, dk)), c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (H,), _F32), float(scale),
          c("S0", S0, (B, H, dk, dv), _F32, True), c("lens", lens, (B,), _I32, True),
          c("o", o, (B, T, H, dv)), c("S_T", S_T, (B, H, dk, dv), _F32, True),
          B, T, H, Hk, dk, dv, c.code, ws, nbytes)


def kda_linear_prefill_paged(q, k, v, g, scale, pool, slots_in, slots_out, o, lens=None,
                             workspace=None, stream=None):
    """C entry point kda_linear_prefill_paged: states from pool[slots_in[b]] into
    pool[slots_out[b]] (either table may be None)."""
    c = _Call("kda_linear_prefill_paged", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_linear_prefill_paged", stream, c("q", q, (B, T, Hk, dk)),
          c("k", k, (B, T, Hk, dk)), c("v", v, (B, T, H, dv)), c("g", g, (H,), _F32),
          float(scale), pp, n_slots, c("slots_in", slots_in, (B,), _I32, True),
          c("slots_out", slots_out, (B,), _I32, True), c("lens", lens, (B,), _I32, True),
          c("o", o, (B, T, H, dv)), B, T, H, Hk, dk, dv, c.code, ws, nbytes)


def linear_prefill(q, k, v, g, scale=1.0, S0=None, lens=None, want_state=True, o=None,
                   stream=None):
    """kda_linear_prefill with S_T, the workspace and (unless given) o allocated;
    an allocated o is zero past the lengths.  Returns (o, S_T or None)."""
    c = _Call("linear_prefill", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    with _on(q, stream):
        if o is None:
            new = torch.empty if lens is None else torch.zeros
            o = new((B, T, H, dv), dtype=q.dtype, device=q.device)
        S_T = torch.empty((B, H, dk, dv), dtype=_F32, device=q.device) if want_state else None
        ws = _empty(lib().kda_linear_prefill_workspace_bytes(B, T, H, Hk, dk, dv, c.code), q.device)
        kda_linear_prefill(q, k, v, g, scale, S0, o, S_T, lens, ws, stream)
    return o, S_T


def kda_linear_backward(q, k, v, g, scale, S0, dO, dS_T, dq, dk, dv, dS0, lens=None,
                        workspace=None, stream=None):
    """C entry point kda_linear_backward."""
    c = _Call("kda_linear_backward", q, 4)
    B, T, H, dvv, Hk, dkk = _dims(c, q, v, 4)
    qk, vo, st = (B, T, Hk, dkk), (B, T, H, dvv), (B, H, dkk, dvv)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_linear_backward", stream, c("q", q, qk), c("k", k, qk), c("v", v, vo),
          c("g", g, (H,), _F32), float(scale), c("S0", S0, st, _F32, True),
          c("lens", lens, (B,), _I32, True), c("dO", dO, vo), c("dS_T", dS_T, st, _F32, True),
          c("dq", dq, qk), c("dk", dk, qk), c("dv", dv, vo), c("dS0", dS0, st, _F32, True),
          B, T, H, Hk, dkk, dvv, c.code, ws, nbytes)


def linear_backward(q, k, v, g, dO, scale=1.0, S0=None, dS_T=None, lens=None, want_dS0=True,
                    dq=None, dk=None, dv=None, stream=None):
    """kda_linear_backward with the workspace and the gradients that are not given
    allocated; allocated ones are zero past the lengths.  Returns a dict with
    dq, dk, dv, dS0."""
    c = _Call("linear_backward", q, 4)
    B, T, H, dvv, Hk, dkk = _dims(c, q, v, 4)
    with _on(q, stream):
        new = torch.empty_like if lens is None else torch.zeros_like
        dq = new(q) if dq is None else dq
        dk = new(q) if dk is None else dk
        dv = new(v) if dv is None else dv
        dS0 = torch.empty((B, H, dkk, dvv), dtype=_F32, device=q.device) if want_dS0 else None
        ws = _empty(lib().kda_linear_backward_workspace_bytes(B, T, H, Hk, dkk, dvv, c.code),
                    q.device)
        kda_linear_backward(q, k, v, g, scale, S0, dO, dS_T, dq, dk, dv, dS0, lens, ws, stream)
    return dict(dq=dq, dk=dk, dv=dv, dS0=dS0)


def kda_linear_decode_step(q, k, v, g, scale, S, o, stream=None):
    """C entry point kda_linear_decode_step; S is updated in place."""
    c = _Call("kda_linear_decode_step", q, 3)
    B, H, dv, Hk, dk = _dims(c, q, v, 3)
    c.run("kda_linear_decode_step", stream, c("q", q, (B, Hk, dk)), c("k", k, (B, Hk, dk)),
          c("v", v, (B, H, dv)), c("g", g, (H,), _F32), float(scale),
          c("S", S, (B, H, dk, dv), _F32), c("o", o, (B, H, dv)), B, H, Hk, dk, dv, c.code)


def kda_linear_decode_step_paged(q, k, v, g, scale, pool, slots, o, stream=None):
    """C entry point kda_linear_decode_step_paged: pool[slots[b]] updated in place."""
    c = _Call("kda_linear_decode_step_paged", q, 3)
    B, H, dv, Hk, dk = _dims(c, q, v, 3)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    c.run("kda_linear_decode_step_paged", stream, c("q", q, (B, Hk, dk)), c("k", k, (B, Hk, dk)),
          c("v", v, (B, H, dv)), c("g", g, (H,), _F32), float(scale), pp, n_slots,
          c("slots", slots, (B,), _I32), c("o", o, (B, H, dv)), B, H, Hk, dk, dv, c.code)


def linear_decode_step(q, k, v, g, S, scale=1.0, stream=None):
    """kda_linear_decode_step with o allocated (S updated in place).  Returns o."""
    with _on(v, stream):
        o = torch.empty_like(v)
        kda_linear_decode_step(q, k, v, g, scale, S, o, stream)
    return o


# ----------------------------------------------------------------- draft trees

def kda_linear_tree(q, k, v, g, scale, S, parent, o, stream=None):
    """C entry point kda_linear_tree; parent int32 [B, T]."""
    c = _Call("kda_linear_tree", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    c.run("kda_linear_tree", stream, c("q", q, (B, T, Hk, dk)), c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (H,), _F32), float(scale),
          c("S", S, (B, H, dk, dv), _F32), c("parent", parent, (B, T), _I32),
          c("o", o, (B, T, H, dv)), B, T, H, Hk, dk, dv, c.code)


def kda_linear_tree_paged(q, k, v, g, scale, pool, slots, parent, o, stream=None):
    """C entry point kda_linear_tree_paged: the states pool[slots[b]]."""
    c = _Call("kda_linear_tree_paged", q, 4)
    B, T, H, dv, Hk, dk = _dims(c, q, v, 4)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    c.run("kda_linear_tree_paged", stream, c("q", q, (B, T, Hk, dk)), c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (H,), _F32), float(scale), pp, n_slots,
          c("slots", slots, (B,), _I32), c("parent", parent, (B, T), _I32),
          c("o", o, (B, T, H, dv)), B, T, H, Hk, dk, dv, c.code)


def linear_tree(q, k, v, g, S, parent, scale=1.0, stream=None):
    """kda_linear_tree with o allocated.  Returns o."""
    with _on(v, stream):
        o = torch.empty_like(v)
        kda_linear_tree(q, k, v, g, scale, S, parent, o, stream)
    return o


def kda_linear_tree_commit(k, v, g, parent, accepted, S, S_out, stream=None):
    """C entry point kda_linear_tree_commit; accepted int32 [B], S_out may be S."""
    c = _Call("kda_linear_tree_commit", k, 4)
    B, T, H, dv, Hk, dk = _dims(c, k, v, 4)
    c.run("kda_linear_tree_commit", stream, c("k", k, (B, T, Hk, dk)), c("v", v, (B, T, H, dv)),
          c("g", g, (H,), _F32), c("parent", parent, (B, T), _I32),
          c("accepted", accepted, (B,), _I32), c("S", S, (B, H, dk, dv), _F32),
          c("S_out", S_out, (B, H, dk, dv), _F32), B, T, H, Hk, dk, dv, c.code)


def kda_linear_tree_commit_paged(k, v, g, parent, accepted, pool, slots_in, slots_out,
                                 stream=None):
    """C entry point kda_linear_tree_commit_paged: from pool[slots_in[b]] into
    pool[slots_out[b]]."""
    c = _Call("kda_linear_tree_commit_paged", k, 4)
    B, T, H, dv, Hk, dk = _dims(c, k, v, 4)
    pp, n_slots = _pool(c, pool, H, dk, dv)
    c.run("kda_linear_tree_commit_paged", stream, c("k", k, (B, T, Hk, dk)),
          c("v", v, (B, T, H, dv)), c("g", g, (H,), _F32), c("parent", parent, (B, T), _I32),
          c("accepted", accepted, (B,), _I32), pp, n_slots,
          c("slots_in", slots_in, (B,), _I32), c("slots_out", slots_out, (B,), _I32),
          B, T, H, Hk, dk, dv, c.code)


def linear_tree_commit(k, v, g, S, parent, accepted, S_out=None, stream=None):
    """kda_linear_tree_commit; without S_out the state is committed in place.
    Returns the state after the accepted path."""
    S_out = S if S_out is None else S_out
    kda_linear_tree_commit(k, v, g, parent, accepted, S, S_out, stream)
    return S_out


# ----------------------------------------------------------------- norm and rotation

def _norm_dims(c, q, k):
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError(f"{c.where}: k must be a tensor with 4 dimensions")
    return (*q.shape[:3], k.shape[2], q.shape[3])


def _rot(c, inv_freq):
    """Elements of a head that are turned: two for each frequency."""
    if inv_freq is None:
        return 0
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError(f"{c.where}: inv_freq must be a tensor [rot / 2]")
    return 2 * inv_freq.shape[0]


def _norm(c, norm):
    if norm not in _NORMS:
        raise ValueError(f"{c.where}: norm must be one of {sorted(_NORMS)}, got {norm!r}")
    return _NORMS[norm]


def kda_qk_norm_rope(q, k, w_q, w_k, positions, inv_freq, norm, eps, interleaved, y_q, y_k,
                     stream=None):
    """C entry point kda_qk_norm_rope; norm "l2" or "rms", positions int32 [B, T],
    inv_freq fp32 [rot / 2] (both None: no rotation), y_q may be q and y_k k."""
    c = _Call("kda_qk_norm_rope", q, 4)
    B, T, H, Hk, d = _norm_dims(c, q, k)
    rot = _rot(c, inv_freq)
    c.run("kda_qk_norm_rope", stream, c("q", q, (B, T, H, d)), c("k", k, (B, T, Hk, d)),
          c("w_q", w_q, (d,), _F32, True), c("w_k", w_k, (d,), _F32, True),
          c("positions", positions, (B, T), _I32, rot == 0),
          c("inv_freq", inv_freq, (rot // 2,), _F32, rot == 0), _norm(c, norm), float(eps), rot,
          int(bool(interleaved)), c("y_q", y_q, (B, T, H, d)), c("y_k", y_k, (B, T, Hk, d)),
          B, T, H, Hk, d, c.code)


def qk_norm_rope(q, k, positions=None, inv_freq=None, w_q=None, w_k=None, norm="rms", eps=1e-6,
                 interleaved=False, stream=None):
    """kda_qk_norm_rope with the outputs allocated.  Returns (y_q, y_k)."""
    with _on(q, stream):
        y_q, y_k = torch.empty_like(q), torch.empty_like(k)
        kda_qk_norm_rope(q, k, w_q, w_k, positions, inv_freq, norm, eps, interleaved, y_q, y_k,
                         stream)
    return y_q, y_k


def kda_qk_norm_rope_backward_workspace_bytes(B, T, H, H_k, d, dtype) -> int:
    return int(lib().kda_qk_norm_rope_backward_workspace_bytes(B, T, H, H_k, d, _code(dtype)))


def kda_qk_norm_rope_backward(q, k, w_q, w_k, positions, inv_freq, norm, eps, interleaved, dy_q,
                              dy_k, dq, dk, dw_q, dw_k, workspace=None, stream=None):
    """C entry point kda_qk_norm_rope_backward; dw_q and dw_k may be None."""
    c = _Call("kda_qk_norm_rope_backward", q, 4)
    B, T, H, Hk, d = _norm_dims(c, q, k)
    rot = _rot(c, inv_freq)
    sq, sk = (B, T, H, d), (B, T, Hk, d)
    ws, nbytes = c.workspace(workspace)
    c.run("kda_qk_norm_rope_backward", stream, c("q", q, sq), c("k", k, sk),
          c("w_q", w_q, (d,), _F32, True), c("w_k", w_k, (d,), _F32, True),
          c("positions", positions, (B, T), _I32, rot == 0),
          c("inv_freq", inv_freq, (rot // 2,), _F32, rot == 0), _norm(c, norm), float(eps), rot,
          int(bool(interleaved)), c("dy_q", dy_q, sq), c("dy_k", dy_k, sk), c("dq", dq, sq),
          c("dk", dk, sk), c("dw_q", dw_q, (d,), _F32, True), c("dw_k", dw_k, (d,), _F32, True),
          B, T, H, Hk, d, c.code, ws, nbytes)


def qk_norm_rope_backward(q, k, positions, inv_freq, dy_q, dy_k, w_q=None, w_k=None, norm="rms",
                          eps=1e-6, interleaved=False, stream=None):
    """kda_qk_norm_rope_backward with the gradients and the workspace allocated.
    Returns a dict with dq, dk, dw_q, dw_k (the last two None without weights)."""
    c = _Call("qk_norm_rope_backward", q, 4)
    B, T, H, Hk, d = _norm_dims(c, q, k)
    with _on(q, stream):
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dw_q, dw_k = (None if w is None else torch.empty(d, dtype=_F32, device=q.device)
                      for w in (w_q, w_k))
        ws = None
        if w_q is not None or w_k is not None:
            ws = _empty(kda_qk_norm_rope_backward_workspace_bytes(B, T, H, Hk, d, q.dtype), q.device)
        kda_qk_norm_rope_backward(q, k, w_q, w_k, positions, inv_freq, norm, eps, interleaved,
                                  dy_q, dy_k, dq, dk, dw_q, dw_k, ws, stream)
    return dict(dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k)
