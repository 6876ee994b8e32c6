"""Refusals of the linear-attention, draft-tree and norm entry points on the CPU:
the C library rejects bad arguments on the host before any HIP call, the binding
tensors that do not fit.  No call here reaches a kernel launch."""
import ctypes
import os
import re

import pytest
import torch

import linear_attention_recurrence_05_amd as kda
from linear_attention_recurrence_05_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kda.h")
E = {n: i for i, n in enumerate(_lib._STATUS)}


def at(i, off=0):
    """A fake device address, never dereferenced: every call below is refused."""
    return ctypes.c_void_p((1 << 40) + i * (1 << 36) + off)


INF = float("inf")
SIZES = dict(B=2, T=64, H=4, H_k=2, d_k=64, d_v=128, dt=kda.KDA_BF16)
WS = dict(workspace=at(30), workspace_bytes=1 << 34, stream=None)
CALLS = {
    "kda_linear_prefill": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, S0=at(4), lens=at(5), o=at(6),
                               S_T=at(7), **SIZES, **WS),
    "kda_linear_prefill_paged": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, pool=at(4), n_slots=3,
                                     slots_in=at(5), slots_out=at(6), lens=at(7), o=at(8), **SIZES, **WS),
    "kda_linear_backward": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, S0=at(4), lens=at(5), dO=at(6),
                                dS_T=at(7), dq=at(8), dk=at(9), dv=at(10), dS0=at(11), **SIZES, **WS),
    "kda_linear_decode_step": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, S=at(4), o=at(5), B=2, H=4,
                                   H_k=2, d_k=64, d_v=128, dt=kda.KDA_BF16, stream=None),
    "kda_linear_decode_step_paged": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, pool=at(4), n_slots=3,
                                         slots=at(5), o=at(6), B=2, H=4, H_k=2, d_k=64, d_v=128,
                                         dt=kda.KDA_BF16, stream=None),
    "kda_linear_tree": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, S=at(4), parent=at(5), o=at(6),
                            **SIZES, stream=None),
    "kda_linear_tree_paged": dict(q=at(0), k=at(1), v=at(2), g=at(3), scale=1.0, pool=at(4), n_slots=3,
                                  slots=at(5), parent=at(6), o=at(7), **SIZES, stream=None),
    "kda_linear_tree_commit": dict(k=at(1), v=at(2), g=at(3), parent=at(5), accepted=at(6), S=at(4), S_out=at(7),
                                   **SIZES, stream=None),
    "kda_linear_tree_commit_paged": dict(k=at(1), v=at(2), g=at(3), parent=at(5), accepted=at(6), pool=at(4),
                                         n_slots=3, slots_in=at(7), slots_out=at(8), **SIZES, stream=None),
    "kda_qk_norm_rope": dict(q=at(0), k=at(1), w_q=at(2), w_k=at(3), positions=at(4), inv_freq=at(5), norm=0,
                             eps=1e-6, rot=64, interleaved=0, y_q=at(6), y_k=at(7), B=2, T=64, H=4, H_k=2, d=64,
                             dt=kda.KDA_BF16, stream=None),
    "kda_qk_norm_rope_backward": dict(q=at(0), k=at(1), w_q=at(2), w_k=at(3), positions=at(4), inv_freq=at(5),
                                      norm=0, eps=1e-6, rot=64, interleaved=0, dy_q=at(6), dy_k=at(7), dq=at(8),
                                      dk=at(9), dw_q=at(10), dw_k=at(11), B=2, T=64, H=4, H_k=2, d=64,
                                      dt=kda.KDA_BF16, **WS),
}
LINEAR = [n for n in CALLS if "linear" in n]
NORM = [n for n in CALLS if "norm" in n]


def refuse(name, code, **over):
    args = dict(CALLS[name])
    assert set(over) <= set(args), (name, over)
    args.update(over)
    L = kda.lib()
    st = getattr(L, name)(*args.values())
    assert st == E[code] and L.kda_last_error().decode(), (name, over, st, L.kda_last_error())


def test_the_argument_lists_are_the_headers():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, args in CALLS.items():
        decl = re.search(r"\b%s\s*\(([^)]*)\)" % name, text).group(1)
        assert [a.split()[-1].lstrip("*") for a in decl.split(",")] == list(args), name


@pytest.mark.parametrize("name", LINEAR)
def test_linear_calls_refuse(name):
    has = CALLS[name]
    for over, code in [
        (dict(B=0), "KDA_ERR_INVALID_SHAPE"), (dict(H=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(H_k=3), "KDA_ERR_INVALID_SHAPE"), (dict(H_k=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(H_k=8), "KDA_ERR_INVALID_SHAPE"), (dict(T=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(B=1 << 26), "KDA_ERR_INVALID_SHAPE"), (dict(B=(1 << 21) + 1, H=4), "KDA_ERR_INVALID_SHAPE"), (dict(H=1 << 18, H_k=1 << 18), "KDA_ERR_INVALID_SHAPE"),
        (dict(d_k=48), "KDA_ERR_UNSUPPORTED"), (dict(d_v=256), "KDA_ERR_UNSUPPORTED"),
        (dict(dt=2), "KDA_ERR_UNSUPPORTED"), (dict(scale=INF), "KDA_ERR_INVALID_VALUE"),
        (dict(scale=float("nan")), "KDA_ERR_INVALID_VALUE"), (dict(n_slots=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(n_slots=1 << 25), "KDA_ERR_INVALID_SHAPE"),
        (dict(workspace=None), "KDA_ERR_NULL_POINTER"), (dict(workspace_bytes=0), "KDA_ERR_WORKSPACE_TOO_SMALL"),
    ]:
        if not set(over) <= set(has):
            continue
        if "workspace" in str(over):
            big = dict(B=1, T=8192, H=2, H_k=1)
            size = getattr(kda, name.replace("_paged", "") + "_workspace_bytes")(1, 8192, 2, 1, 64, 128, kda.KDA_BF16)
            if size:
                refuse(name, code, **over, **big)
            continue
        refuse(name, code, **over)
    for p in ("q", "k", "v", "g", "o", "S", "pool", "dO", "dq", "dk", "dv", "parent", "accepted", "slots", "S_out"):
        if p in has:
            refuse(name, "KDA_ERR_NULL_POINTER", **{p: None})
            refuse(name, "KDA_ERR_MISALIGNED", **{p: ctypes.c_void_p(has[p].value + 2)})
    for p in ("S0", "S_T", "dS_T", "dS0"):
        if p in has:
            refuse(name, "KDA_ERR_MISALIGNED", **{p: ctypes.c_void_p(has[p].value + 4)})
    for out in ("o", "S_T", "S_out", "dq", "dk", "dv", "dS0"):
        for p in ("k", "v", "g", "parent", "lens"):
            if out in has and p in has:
                refuse(name, "KDA_ERR_ALIASING", **{out: has[p]})
    for out, src in (("S_T", "S0"), ("S_out", "S")):
        if out in has and src in has:                     # in place is fine, a partial overlap is not
            refuse(name, "KDA_ERR_ALIASING", **{out: ctypes.c_void_p(has[src].value + 16)})
    if "pool" in has and "o" in has:
        refuse(name, "KDA_ERR_ALIASING", o=ctypes.c_void_p(has["pool"].value + 64))
    if "tree" in name:
        refuse(name, "KDA_ERR_INVALID_SHAPE", T=65)


@pytest.mark.parametrize("name", NORM)
def test_norm_calls_refuse(name):
    has = CALLS[name]
    for over, code in [
        (dict(B=0), "KDA_ERR_INVALID_SHAPE"), (dict(T=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(H=0), "KDA_ERR_INVALID_SHAPE"), (dict(H_k=0), "KDA_ERR_INVALID_SHAPE"),
        (dict(d=96), "KDA_ERR_UNSUPPORTED"), (dict(dt=-1), "KDA_ERR_UNSUPPORTED"),
        (dict(norm=2), "KDA_ERR_INVALID_VALUE"), (dict(eps=0.0), "KDA_ERR_INVALID_VALUE"),
        (dict(eps=-1.0), "KDA_ERR_INVALID_VALUE"), (dict(eps=INF), "KDA_ERR_INVALID_VALUE"),
        (dict(eps=float("nan")), "KDA_ERR_INVALID_VALUE"), (dict(rot=65), "KDA_ERR_INVALID_VALUE"),
        (dict(rot=66), "KDA_ERR_INVALID_VALUE"), (dict(rot=-2), "KDA_ERR_INVALID_VALUE"),
        (dict(interleaved=2), "KDA_ERR_INVALID_VALUE"), (dict(positions=None), "KDA_ERR_NULL_POINTER"),
        (dict(inv_freq=None), "KDA_ERR_NULL_POINTER"),
    ]:
        refuse(name, code, **over)
    for p in ("q", "k", "y_q", "y_k", "dy_q", "dy_k", "dq", "dk"):
        if p in has:
            refuse(name, "KDA_ERR_NULL_POINTER", **{p: None})
            refuse(name, "KDA_ERR_MISALIGNED", **{p: ctypes.c_void_p(has[p].value + 8)})
    if name.endswith("backward"):
        refuse(name, "KDA_ERR_ALIASING", dq=has["q"])
        refuse(name, "KDA_ERR_ALIASING", dq=has["dy_k"])
        refuse(name, "KDA_ERR_ALIASING", dw_q=has["w_q"])
        refuse(name, "KDA_ERR_NULL_POINTER", w_q=None)              # dw_q without w_q
        refuse(name, "KDA_ERR_NULL_POINTER", workspace=None)
        refuse(name, "KDA_ERR_WORKSPACE_TOO_SMALL", workspace_bytes=8)
    else:
        refuse(name, "KDA_ERR_ALIASING", y_q=ctypes.c_void_p(has["q"].value + 16))
        refuse(name, "KDA_ERR_ALIASING", y_q=has["k"])
        refuse(name, "KDA_ERR_ALIASING", y_k=has["y_q"])


def test_workspace_queries_of_refused_sizes_are_zero():
    for name in ("kda_linear_prefill_workspace_bytes", "kda_linear_backward_workspace_bytes"):
        f = getattr(kda, name)
        assert f(0, 64, 4, 2, 64, 64, kda.KDA_BF16) == 0
        assert f(1, 64, 4, 3, 64, 64, kda.KDA_BF16) == 0
        assert f(1, 64, 4, 2, 96, 64, kda.KDA_BF16) == 0
        assert f(1, 64, 4, 2, 64, 64, 5) == 0
    assert kda.kda_linear_backward_workspace_bytes(2, 64, 4, 2, 64, 64, torch.bfloat16) > 0
    f = kda.kda_qk_norm_rope_backward_workspace_bytes
    assert f(1, 0, 4, 2, 64, kda.KDA_BF16) == 0 and f(1, 64, 4, 2, 48, kda.KDA_BF16) == 0
    assert f(1, 64, 4, 2, 64, kda.KDA_BF16) > 0


# ----------------------------------------------------------------- the binding

def tensors(dtype=torch.bfloat16):
    B, T, H, Hk, dk, dv = 2, 6, 4, 2, 32, 64
    z = torch.zeros
    return dict(q=z(B, T, Hk, dk, dtype=dtype), k=z(B, T, Hk, dk, dtype=dtype), v=z(B, T, H, dv, dtype=dtype),
                g=z(H), S=z(B, H, dk, dv), o=z(B, T, H, dv, dtype=dtype),
                parent=z(B, T, dtype=torch.int32), accepted=z(B, dtype=torch.int32),
                lens=z(B, dtype=torch.int32))


def calls(x):
    yield lambda: kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], 1.0, x["S"], x["lens"], o=x["o"])
    yield lambda: kda.linear_backward(x["q"], x["k"], x["v"], x["g"], x["o"], 1.0, x["S"], x["S"], x["lens"])
    yield lambda: kda.linear_tree(x["q"], x["k"], x["v"], x["g"], x["S"], x["parent"])
    yield lambda: kda.linear_tree_commit(x["k"], x["v"], x["g"], x["S"], x["parent"], x["accepted"])


def test_the_binding_refuses_host_tensors():
    for call in calls(tensors()):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.parametrize("name,bad,error", [
    ("k", lambda t: t.float(), ValueError), ("k", lambda t: t[:, :, :1], ValueError),
    ("k", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
    ("v", lambda t: t[:, :5], ValueError), ("v", lambda t: t[0], ValueError), ("v", lambda t: None, (TypeError, ValueError)),
    ("g", lambda t: t.double(), ValueError), ("g", lambda t: t[:3], ValueError),
    ("S", lambda t: t.bfloat16(), ValueError), ("S", lambda t: t.transpose(2, 3), ValueError),
    ("k", lambda t: "k", (TypeError, ValueError)),
])
def test_the_binding_refuses_tensors_that_do_not_fit(monkeypatch, name, bad, error):
    monkeypatch.setattr(_lib, "_DEVICE_TYPE", "cpu")
    x = tensors()
    x[name] = bad(x[name])
    for call in calls(x):
        with pytest.raises(error):
            call()


def test_the_binding_refuses_tables_norms_and_dtypes(monkeypatch):
    monkeypatch.setattr(_lib, "_DEVICE_TYPE", "cpu")
    x = tensors()
    for name in ("parent", "accepted", "lens"):
        y = {**x, name: x[name].long()}
        with pytest.raises(ValueError, match=name):
            list(c() for i, c in enumerate(calls(y)) if (name == "lens") == (i < 2) and (name != "accepted" or i == 3))
    y = {n: t.half() if t.dtype == torch.bfloat16 else t for n, t in x.items()}
    for call in calls(y):
        with pytest.raises(ValueError, match="bfloat16 or float32"):
            call()
    q, k, pos, f = x["v"], x["v"][:, :, :2].contiguous(), x["parent"], torch.zeros(16)
    for kw, match in ((dict(norm="max"), "norm"), (dict(w_q=torch.zeros(63)), "w_q"), (dict(w_k=torch.zeros(64).half()), "w_k"),
                      (dict(positions=pos.long()), "positions"), (dict(positions=None), "positions"),
                      (dict(inv_freq=f.double()), "inv_freq"), (dict(k=k[..., :32].contiguous()), "k has shape")):
        args = {**dict(q=q, k=k, positions=pos, inv_freq=f), **kw}
        with pytest.raises(ValueError, match=match):
            kda.qk_norm_rope(**args)


def test_more_sequences_than_a_launch_holds_are_refused():
    for name in LINEAR:
        refuse(name, "KDA_ERR_INVALID_SHAPE", B=(1 << 20) + 1, H=4, **({"T": 1} if "T" in CALLS[name] else {}))
    for f in (kda.kda_linear_prefill_workspace_bytes, kda.kda_linear_backward_workspace_bytes):
        assert f((1 << 22) + 1, 1, 1, 1, 32, 32, kda.KDA_BF16) == 0
        assert f(1 << 22, 65, 1, 1, 128, 128, kda.KDA_BF16) == 0       # one segment: three workgroups each


def test_in_place_outputs_refuse_a_second_input_at_the_same_address():
    """The output may be the input it replaces, not another one that shares its memory."""
    same = dict(H=4, H_k=4)
    refuse("kda_qk_norm_rope", "KDA_ERR_ALIASING", k=at(0), y_q=at(0), **same)
    refuse("kda_qk_norm_rope", "KDA_ERR_ALIASING", k=at(0), y_k=at(0), **same)
    refuse("kda_qk_norm_rope_backward", "KDA_ERR_ALIASING", dy_k=at(6), dq=at(6), **same)
    refuse("kda_qk_norm_rope_backward", "KDA_ERR_ALIASING", q=at(6), dq=at(6))
    sizes = dict(B=1, H=1, H_k=1, T=32, d_k=32, d_v=32, dt=kda.KDA_F32)     # q, v and a state: the same bytes
    refuse("kda_linear_prefill", "KDA_ERR_ALIASING", S_T=at(4), v=at(4), **sizes)
    refuse("kda_linear_tree_commit", "KDA_ERR_ALIASING", S_out=at(4), v=at(4), **sizes)
