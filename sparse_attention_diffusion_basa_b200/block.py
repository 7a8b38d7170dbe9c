"""The rows of a Diffusion Transformer block around its attention: RMS norm and
rotary positions of q and k between the projection and the attention calls, and
the border between two blocks (branch norm, gate, residual, next norm and
modulation), each with its backward.

Argument marshalling only, as in the rest of the binding: the computation runs
in the library's CUDA kernels.  A call runs on the current stream of its
tensors' device, or on ``stream``; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import (BASA_BF16, BASA_F32, BASA_FP8_E4M3, BASA_NORM, BASA_ROPE_LAYOUT, BASA_ROPE_NORM,
                   BasaGnormParams, BasaRopeParams)

_DT = {torch.float32: BASA_F32, torch.bfloat16: BASA_BF16, torch.float8_e4m3fn: BASA_FP8_E4M3}
_FLOAT = (torch.float32, torch.bfloat16)
_E4M3 = torch.float8_e4m3fn

# The small calls of a sampler are bound by this file, not by their kernels, so
# the checks of a call's shapes, strides, types and devices and the parameter
# struct they lead to are kept (lru_cache) by just these and by the numbers given,
# as Python numbers: never by a tensor, its address or its values.  A factor held in
# a 0-dim tensor hashes by identity, so numbers are converted ahead of the lookup.
_KEPT = 512


def _meta(t):
    """What the checks look at: (shape, strides, dtype, device), or None."""
    if t is None:
        return None
    try:
        return t.shape, t.stride(), t.dtype, t.device
    except AttributeError:
        raise TypeError(f"expected a torch tensor, got {type(t).__name__}") from None


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _code(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {key!r}") from None


def _three(xs, name, kind):
    """Three numbers as Python numbers of ``kind``."""
    try:
        a, b, c = xs
    except ValueError:
        raise ValueError(f"{name} must give three values, got {xs}") from None
    if type(a) is kind and type(b) is kind and type(c) is kind:
        return a, b, c
    return kind(a), kind(b), kind(c)


def _given(stream, device):
    """``stream`` as the current one, for tensors on ``device`` (a tensor's, or None: not known here)."""
    if device is not None and device.type == "cuda" and device != stream.device:
        raise ValueError(f"stream is one of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _device(*tensors):
    """The device of the first tensor there is."""
    return next((t.device for t in tensors if isinstance(getattr(t, "device", None), torch.device)), None)


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _on(device, fn, what: str, *args):
    """Calls ``fn`` with ``device`` current and its current stream as the last argument."""
    index = device.index
    if torch.cuda.current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        _lib.check(code, what)


@functools.lru_cache(maxsize=_KEPT)
def _size(device, name, ref) -> int:
    """Workspace bytes for a plan's struct, asked with ``device`` current (they go by its SMs)."""
    with torch.cuda.device(device.index):
        return int(getattr(_lib.load(), name)(ref.params))


def _like(t, dtype=None):
    """A dense tensor of t's shape (half the host time of torch.empty with a shape)."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _workspace(device, need, workspace):
    if not need:
        return None
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} contiguous bytes on {device}")
    return workspace


class _Plan:
    """A checked call: its parameter struct (as passed) and what the call allocates by."""

    def __init__(self, struct, **kw):
        self.struct, self.params = struct, ctypes.byref(struct)
        self.__dict__.update(kw)


def _tensor(m, ref, name, dtypes):
    if m is None:
        raise TypeError(f"{name} must be a torch tensor")
    if m[3].type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if ref is not None and m[3] != ref[3]:
        raise ValueError(f"{name} must be on {ref[3]}, got {m[3]}")
    if m[2] not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {m[2]}")


def _numel(shape):
    n = 1
    for s in shape:
        n *= s
    return n


def _dense(m) -> bool:
    expect = 1
    for size, st in zip(reversed(m[0]), reversed(m[1])):
        if size != 1:
            if st != expect:
                return _numel(m[0]) == 0
            expect *= size
    return True


def _row_stride(shape, stride, n, name) -> int:
    """Elements between consecutive rows when the first n dims are walked in order."""
    ld = expect = None
    for size, st in zip(reversed(shape[:n]), reversed(stride[:n])):
        if size == 1:
            continue
        if ld is None:
            ld = st
        elif st != expect:
            raise ValueError(f"the rows of {name} {tuple(shape)} must lie at one stride, got {tuple(stride)}: "
                             "make it contiguous")
        expect = st * size
    return ld


# ---------------------------------------------------------------------------
# q/k/v preparation
# ---------------------------------------------------------------------------
def _heads(m, ref, name, dtypes, dense=False) -> int:
    """Checks a [B, T, Hg, Wg, heads, d] (or text [B, L, heads, d]) tensor; its row stride, 0 = dense."""
    _tensor(m, ref, name, dtypes)
    shape, stride = m[0], m[1]
    if len(shape) not in (4, 6):
        raise ValueError(f"{name} must be [B, T, Hg, Wg, heads, d] or [B, L, heads, d], got {tuple(shape)}")
    if _dense(m):
        return 0
    if dense:
        raise ValueError(f"{name} must be contiguous")
    if (shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1]):
        raise ValueError(f"the heads of {name} must be dense, got strides {tuple(stride)}")
    ld = _row_stride(shape, stride, len(shape) - 2, name)
    if ld is None:
        return 0
    if ld < shape[-1] * shape[-2]:
        raise ValueError(f"the rows of {name} overlap: strides {tuple(stride)}")
    return ld


def _rope_params(q, k, axes, layout, norm, eps, out_dtype, descale, lds, w_dtype) -> BasaRopeParams:
    q, k, dtype = q[0], k[0], q[2]
    if k[:-2] != q[:-2] or k[-1] != q[-1]:
        raise ValueError(f"k {tuple(k)} must match q {tuple(q)} except in heads")
    H, Hkv = q[-2], k[-2]
    if H != Hkv and (H == 0 or Hkv == 0 or H % Hkv):
        raise ValueError(f"q heads {H} must be a multiple of k/v heads {Hkv}")
    T, Hg, Wg = q[1:4] if len(q) == 6 else (1, 1, q[1])
    at, ah, aw = axes
    return BasaRopeParams(q[0], H, Hkv, T, Hg, Wg, q[-1], at, ah, aw, _code(BASA_ROPE_LAYOUT, layout, "layout"),
                          _code(BASA_ROPE_NORM, norm, "norm"), eps, _DT[dtype], _DT[out_dtype],
                          _DT[w_dtype], *descale, *lds)


def _pairs(prm) -> int:
    return prm.T * (prm.at // 2) + prm.Hg * (prm.ah // 2) + prm.Wg * (prm.aw // 2)


def _check_table(table, q, prm) -> bool:
    """Whether the call turns anything; then the table has to fit."""
    n = _pairs(prm)
    if n == 0:
        return False
    _tensor(table, q, "table", (torch.float32,))
    if _numel(table[0]) != 2 * n or not _dense(table):
        raise ValueError(f"table must hold {n} contiguous (cos, sin) pairs for this grid and these axes, "
                         f"got {tuple(table[0])}")
    return True


def _weights(q, k, q_weight, k_weight, norm):
    """Checks the norm weights; their dtype."""
    dtype = None
    for w, t, name in ((q_weight, q, "q_weight"), (k_weight, k, "k_weight")):
        if w is None:
            continue
        if norm is None:
            raise ValueError(f"{name} needs a norm")
        _tensor(w, q, name, _FLOAT)
        n = t[0][-1] * (t[0][-2] if norm == "token" else 1)
        if _numel(w[0]) != n or not _dense(w):
            raise ValueError(f"{name} must be {n} contiguous values, got {tuple(w[0])}")
        if dtype not in (None, w[2]):
            raise TypeError("q_weight and k_weight must share a dtype")
        dtype = w[2]
    return dtype or torch.float32


@functools.lru_cache(maxsize=_KEPT)
def _table_plan(grid, axes, out):
    (T, Hg, Wg), (at, ah, aw) = grid, axes
    d = 32
    while d < at + ah + aw and d < 128:
        d *= 2
    prm = BasaRopeParams(1, 1, 1, T, Hg, Wg, d, at, ah, aw, 0, 0, 1.0, BASA_F32, BASA_F32, BASA_F32)
    if out is not None:
        _check_table(out, out, prm)
    return _Plan(prm, pairs=max(_pairs(prm), 0))


def rope_table(grid, axes, theta: float = 10000.0, start=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0),
               device=None, out=None, stream=None) -> torch.Tensor:
    """The (cos, sin) pairs of a grid (T, Hg, Wg) for ``axes`` = rotated elements of a
    head per axis -> fp32 [T*at/2 + Hg*ah/2 + Wg*aw/2, 2].

    Coordinate i of an axis stands at position start + step * i; pair j turns by
    position * theta^(-2j / width).  Keep it while grid and positions stay."""
    if stream is not None:
        asked = None if device is None else torch.device(device)
        with _given(stream, _device(out) or (asked if asked is not None and asked.index is not None else None)):
            return rope_table(grid, axes, theta, start, step, device, out)
    plan = _table_plan(_three(grid, "grid", int), _three(axes, "axes", int), _meta(out))
    if out is None:
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("device must be a CUDA device")
        out = torch.empty((plan.pairs, 2), dtype=torch.float32, device=dev)
    d3 = ctypes.c_double * 3
    _on(out.device, _lib.load().basa_rope_table, "basa_rope_table", out.data_ptr(), float(theta),
        d3(*_three(start, "start", float)), d3(*_three(step, "step", float)), plan.params)
    return out


@functools.lru_cache(maxsize=_KEPT)
def _rope_plan(q, k, v, q_weight, k_weight, table, out, axes, layout, norm, eps, out_dtype, descale):
    lds = [_heads(q, None, "q", _FLOAT), _heads(k, q, "k", (q[2],)), 0]
    if v is not None:
        lds[2] = _heads(v, q, "v", (q[2],))
        if v[0] != k[0]:
            raise ValueError("k and v must have the same shape")
    dt = q[2] if out_dtype is None else out_dtype
    if dt not in (q[2], _E4M3):
        raise TypeError(f"out_dtype must be {q[2]} or {_E4M3}, got {dt}")
    w_dtype = _weights(q, k, q_weight, k_weight, norm)
    prm = _rope_params(q, k, axes, layout, norm, eps, dt, descale, lds, w_dtype)
    turns = _check_table(table, q, prm)
    if out is not None:
        for o, t, name in zip(out, (q, k, v), "qkv"):
            if (o is None) != (t is None):
                raise ValueError(f"out must give {name}'s output exactly when {name} is given")
            if o is not None:
                _heads(o, q, f"{name}'s output", (dt,), dense=True)
                if o[0] != t[0]:
                    raise ValueError(f"{name}'s output must have shape {tuple(t[0])}")
    return _Plan(prm, dtype=dt, turns=turns)


def qkv_rope(q, k, v=None, table=None, axes=(0, 0, 0), *, layout="pairs", norm=None, q_weight=None,
             k_weight=None, eps=1e-6, out_dtype=None, descale=(0.0, 0.0, 0.0), out=None, stream=None):
    """From a q/k/v projection to the attention's inputs -> (q, k, v), dense.

    RMS norm of q and k (``norm``: None, "head" over each head with weights [d],
    "token" over all heads with weights [H*d], [Hkv*d]), rotary positions with
    ``axes`` rotated elements for time, rows and columns (``table`` from
    rope_table; ``layout`` "pairs": elements 2j, 2j+1; "halves": j, j + sum/2),
    and v (or None) copied along.  q, k, v are [B, T, Hg, Wg, heads, d] (text:
    [B, L, heads, d], grid (1, 1, L)), dense or slices of one projection output.
    ``out_dtype`` torch.float8_e4m3fn writes e4m3 values whose factors are
    ``descale`` (0 = 1), as window_attn takes them.  ``out`` gives the outputs; an
    output may be its own dense input; outputs that overlap otherwise are refused."""
    if stream is not None:
        with _given(stream, _device(q)):
            return qkv_rope(q, k, v, table, axes, layout=layout, norm=norm, q_weight=q_weight, k_weight=k_weight,
                            eps=eps, out_dtype=out_dtype, descale=descale, out=out)
    outs = None if out is None else tuple(_meta(o) for o in out)
    plan = _rope_plan(_meta(q), _meta(k), _meta(v), _meta(q_weight), _meta(k_weight), _meta(table), outs,
                      _three(axes, "axes", int), layout, norm, float(eps), out_dtype,
                      _three(descale, "descale", float))
    dev = q.device
    if out is None:
        dt = plan.dtype
        qo, ko, vo = _like(q, dt), _like(k, dt), None if v is None else _like(v, dt)
    else:
        qo, ko, vo = out
    _on(dev, _lib.load().basa_qkv_rope, "basa_qkv_rope", q.data_ptr(), k.data_ptr(), _p(v), _p(q_weight),
        _p(k_weight), table.data_ptr() if plan.turns else None, qo.data_ptr(), ko.data_ptr(), _p(vo), plan.params)
    return qo, ko, vo


@functools.lru_cache(maxsize=_KEPT)
def _rope_bwd_plan(dq_out, dk_out, dv_out, q, k, q_weight, k_weight, table, out, axes, layout, norm, eps):
    _heads(dq_out, None, "dq_out", _FLOAT, dense=True)
    dtypes = (dq_out[2],)
    _heads(dk_out, dq_out, "dk_out", dtypes, dense=True)
    lds = [0] * 6
    for i, (t, g, name) in enumerate(((q, dq_out, "q"), (k, dk_out, "k"))):
        if norm is None and t is None:
            continue
        lds[i] = _heads(t, dq_out, name, dtypes)
        if t[0] != g[0]:
            raise ValueError(f"{name} {tuple(t[0])} must have the shape of its output's gradient {tuple(g[0])}")
    if dv_out is not None:
        _heads(dv_out, dq_out, "dv_out", dtypes, dense=True)
        if dv_out[0] != dk_out[0]:
            raise ValueError("dk_out and dv_out must have the same shape")
    if out is not None:
        for i, (o, g) in enumerate(zip(out, (dq_out, dk_out, dv_out))):
            if (o is None) != (g is None):
                raise ValueError("out must give dv exactly when dv_out is given")
            if o is not None:
                lds[3 + i] = _heads(o, dq_out, "a gradient", dtypes)
                if o[0] != g[0]:
                    raise ValueError(f"a gradient must have shape {tuple(g[0])}, got {tuple(o[0])}")
    w_dtype = _weights(dq_out, dk_out, q_weight, k_weight, norm)
    prm = _rope_params(dq_out, dk_out, axes, layout, norm, eps, dq_out[2], (0.0, 0.0, 0.0), lds, w_dtype)
    turns = _check_table(table, dq_out, prm)
    return _Plan(prm, turns=turns)


def qkv_rope_bwd(dq_out, dk_out, dv_out, q, k, table=None, axes=(0, 0, 0), *, layout="pairs", norm=None,
                 q_weight=None, k_weight=None, eps=1e-6, out=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dq_weight, dk_weight) of qkv_rope; None for what the call had not.

    ``dq_out``, ``dk_out``, ``dv_out`` (or None) are the dense gradients of its
    outputs, q and k its inputs.  ``out`` = (dq, dk, dv) gives the tensors to
    write, which may be slices of one buffer (dq may be dq_out, and so on)."""
    if stream is not None:
        with _given(stream, _device(dq_out)):
            return qkv_rope_bwd(dq_out, dk_out, dv_out, q, k, table, axes, layout=layout, norm=norm,
                                q_weight=q_weight, k_weight=k_weight, eps=eps, out=out, workspace=workspace)
    outs = None if out is None else tuple(_meta(o) for o in out)
    plan = _rope_bwd_plan(_meta(dq_out), _meta(dk_out), _meta(dv_out), _meta(q), _meta(k), _meta(q_weight),
                          _meta(k_weight), _meta(table), outs, _three(axes, "axes", int), layout, norm, float(eps))
    dev = dq_out.device
    if out is None:
        dq, dk, dv = _like(dq_out), _like(dk_out), None if dv_out is None else _like(dv_out)
    else:
        dq, dk, dv = out
    dqw = None if q_weight is None else _like(q_weight)
    dkw = None if k_weight is None else _like(k_weight)
    ws = None
    if dqw is not None or dkw is not None:
        ws = _workspace(dev, _size(dev, "basa_qkv_rope_bwd_workspace_size", plan), workspace)
    _on(dev, _lib.load().basa_qkv_rope_bwd, "basa_qkv_rope_bwd", dq_out.data_ptr(), dk_out.data_ptr(), _p(dv_out),
        None if norm is None else q.data_ptr(), None if norm is None else k.data_ptr(), _p(q_weight), _p(k_weight),
        table.data_ptr() if plan.turns else None, dq.data_ptr(), dk.data_ptr(), _p(dv), _p(dqw), _p(dkw), _p(ws),
        plan.params)
    return dq, dk, dv, dqw, dkw


# ---------------------------------------------------------------------------
# The border between two blocks
# ---------------------------------------------------------------------------
class GatedNormGrads(NamedTuple):
    """Gradients of gated_norm; None for what the call had not."""
    dx: torch.Tensor
    dy: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]
    dshift: Optional[torch.Tensor]


def _rows(m, ref, name, dtypes, shape=None):
    _tensor(m, ref, name, dtypes)
    if not _dense(m):
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and m[0] != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(m[0])}")


def _modulation(m, x, name):
    """(rows of a modulation, elements from one to the next; 0: one for all)."""
    _tensor(m, x, name, _FLOAT)
    shape, stride, xs = m[0], m[1], x[0]
    C = xs[-1]
    lead = tuple(shape[:-1])
    if len(shape) < 1 or shape[-1] != C or (C > 1 and stride[-1] != 1):
        raise ValueError(f"{name} must end in {C} dense columns, got {tuple(shape)}")
    n = len(lead)
    if n and lead != tuple(xs[:n]) and not (
            n == 2 and len(xs) == 3 and lead[0] == xs[0] and lead[1] and xs[1] % lead[1] == 0):
        raise ValueError(f"{name} {tuple(shape)} must be [C], or lead with dims of x {tuple(xs)}")
    if _numel(lead) == 0:
        return 0, 0
    return _numel(lead), _row_stride(shape, stride, n, name) or 0


def _gnorm_params(x, y_dtype, mods, weights, norm, post_norm, eps, post_eps, res_scale) -> BasaGnormParams:
    """mods: (gate, scale, shift); weights: (post_weight, weight, bias)."""
    C = x[0][-1]
    groups, lds, mod_dtype, w_dtype = None, [], None, None
    for m, name in zip(mods, ("gate", "scale", "shift")):
        if m is None:
            lds.append(0)
            continue
        g, ld = _modulation(m, x, name)
        if groups not in (None, g):
            raise ValueError("gate, scale and shift must have the same leading dims "
                             "(expand the shorter and make it contiguous)")
        if mod_dtype not in (None, m[2]):
            raise TypeError("gate, scale and shift must share a dtype")
        groups, mod_dtype = g, m[2]
        lds.append(ld)
    for w, name in zip(weights, ("post_weight", "weight", "bias")):
        if w is None:
            continue
        _rows(w, x, name, _FLOAT)
        if _numel(w[0]) != C:
            raise ValueError(f"{name} must be {C} values, got {tuple(w[0])}")
        if w_dtype not in (None, w[2]):
            raise TypeError("weight, bias and post_weight must share a dtype")
        w_dtype = w[2]
    return BasaGnormParams(_numel(x[0][:-1]), max(groups or 1, 1), C, _code(BASA_NORM, norm, "norm"),
                           _code(BASA_NORM, post_norm, "post_norm"), eps, post_eps, res_scale,
                           _DT[x[2]], _DT[y_dtype], _DT[mod_dtype or torch.float32],
                           _DT[w_dtype or torch.float32], *lds)


@functools.lru_cache(maxsize=_KEPT)
def _gnorm_plan(x, y, mods, weights, x_out, h_out, norm, post_norm, eps, post_eps, res_scale, h_dtype):
    _rows(x, None, "x", _FLOAT)
    if len(x[0]) < 2:
        raise ValueError(f"x must be [..., C], got {tuple(x[0])}")
    if y is not None:
        _rows(y, x, "y", _FLOAT, x[0])
        if h_dtype not in (None, y[2]):
            raise TypeError(f"h has y's dtype {y[2]}")
        dt = y[2]
    else:
        if mods[0] is not None or post_norm is not None or x_out is not None or norm is None:
            raise ValueError("without y there is no gate, post_norm or x_out, and norm must be given")
        if res_scale != 1.0:
            raise ValueError("res_scale needs y")
        dt = h_dtype or x[2]
        if dt not in _FLOAT:
            raise TypeError(f"h_dtype must be {' or '.join(map(str, _FLOAT))}, got {dt}")
    if norm is None and h_out is not None:
        raise ValueError("h_out needs a norm")
    prm = _gnorm_params(x, dt, mods, weights, norm, post_norm, eps, post_eps, res_scale)
    if x_out is not None:
        _rows(x_out, x, "x_out", (x[2],), x[0])
    if h_out is not None:
        _rows(h_out, x, "h_out", (dt,), x[0])
    return _Plan(prm, dtype=dt, stats=(*x[0][:-1], 4))


def gated_norm(x, y=None, *, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None,
               norm="layer", post_norm=None, eps=1e-6, post_eps=1e-6, res_scale=1.0, h_dtype=None,
               return_stats=False, x_out=None, h_out=None, stream=None):
    """The border between two blocks -> (x_out, h) or (x_out, h, stats):

        x_out = res_scale * x + gate * (post_norm(y) * post_weight)
        h     = (norm(x_out) * weight + bias) * (1 + scale) + shift

    x: residual stream [B, ..., C] (fp32 or bf16), y: the branch's output (x's
    dtype, or bf16 beside an fp32 x); h has y's dtype (without y: ``h_dtype``, by
    default x's).  ``norm``, ``post_norm``: "layer", "rms" or None.  gate, scale,
    shift: [C], [B, C], [B, T, C], ... (one row for the tokens that share the
    leading dims), dense or slices of one modulation output; weight, bias,
    post_weight: [C].  None leaves a part out: y None gives h of x alone (x_out is
    x), norm None gives x_out alone (h is None).  stats (fp32 [B, ..., 4]) is what
    gated_norm_bwd wants.  ``x_out`` may be x, ``h_out`` may be y."""
    if stream is not None:
        with _given(stream, _device(x)):
            return gated_norm(x, y, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                              shift=shift, norm=norm, post_norm=post_norm, eps=eps, post_eps=post_eps,
                              res_scale=res_scale, h_dtype=h_dtype, return_stats=return_stats, x_out=x_out,
                              h_out=h_out)
    plan = _gnorm_plan(_meta(x), _meta(y), (_meta(gate), _meta(scale), _meta(shift)),
                       (_meta(post_weight), _meta(weight), _meta(bias)), _meta(x_out), _meta(h_out), norm, post_norm,
                       float(eps), float(post_eps), float(res_scale), h_dtype)
    dev = x.device
    if x_out is None and y is not None:
        x_out = _like(x)
    if h_out is None and norm is not None:
        h_out = _like(x, plan.dtype)
    stats = torch.empty(plan.stats, dtype=torch.float32, device=dev) if return_stats else None
    _on(dev, _lib.load().basa_gated_norm, "basa_gated_norm", x.data_ptr(), _p(y), _p(gate), _p(post_weight),
        _p(weight), _p(bias), _p(scale), _p(shift), _p(x_out), _p(h_out), _p(stats), plan.params)
    if y is None:
        x_out = x
    return (x_out, h_out, stats) if return_stats else (x_out, h_out)


@functools.lru_cache(maxsize=_KEPT)
def _gnorm_bwd_plan(dh, x_out, stats, y, dx_out, mods, weights, norm, post_norm, res_scale):
    ref = x_out if x_out is not None else dx_out
    _rows(ref, None, "x_out" if x_out is not None else "dx_out", _FLOAT)
    if len(ref[0]) < 2:
        raise ValueError(f"x_out must be [..., C], got {tuple(ref[0])}")
    if (dh is None) != (norm is None):
        raise ValueError("dh goes with a norm")
    if norm is not None and x_out is None:
        raise ValueError("x_out is needed with a norm")
    if norm is None and dx_out is None:
        raise ValueError("dx_out is needed without a norm")
    if y is None and (mods[0] is not None or post_norm is not None or norm is None):
        raise ValueError("without y there is no gate or post_norm, and norm must be given")
    if y is None and res_scale != 1.0:
        raise ValueError("res_scale needs y")
    dt = dh[2] if dh is not None else y[2]
    if dh is not None:
        _rows(dh, ref, "dh", _FLOAT, ref[0])
    if y is not None:
        _rows(y, ref, "y", (dt,), ref[0])
    if dx_out is not None:
        _rows(dx_out, ref, "dx_out", (ref[2],), ref[0])
    use_stats = norm is not None or post_norm is not None
    if use_stats:
        _rows(stats, ref, "stats", (torch.float32,), torch.Size((*ref[0][:-1], 4)))
    prm = _gnorm_params(ref, dt, mods, weights, norm, post_norm, 1.0, 1.0, res_scale)
    return _Plan(prm, use_stats=use_stats, use_y=mods[0] is not None or post_norm is not None)


def gated_norm_bwd(dh, x_out, stats, y=None, dx_out=None, *, gate=None, post_weight=None, weight=None, bias=None,
                   scale=None, shift=None, norm="layer", post_norm=None, res_scale=1.0, workspace=None, stream=None
                   ) -> GatedNormGrads:
    """Gradients of gated_norm for the gradients ``dh`` and ``dx_out`` (or None: zero) of its outputs.

    x_out and stats are the forward's (for a call without y, x_out is x); y and
    the rest as the forward was given them (shift's values are not read).  norm
    None: dh is None and dx_out is required.  dgate, dscale, dshift have the
    modulations' leading dims, dense."""
    if stream is not None:
        with _given(stream, _device(x_out, dx_out)):
            return gated_norm_bwd(dh, x_out, stats, y, dx_out, gate=gate, post_weight=post_weight, weight=weight,
                                  bias=bias, scale=scale, shift=shift, norm=norm, post_norm=post_norm,
                                  res_scale=res_scale, workspace=workspace)
    plan = _gnorm_bwd_plan(_meta(dh), _meta(x_out), _meta(stats), _meta(y), _meta(dx_out),
                           (_meta(gate), _meta(scale), _meta(shift)),
                           (_meta(post_weight), _meta(weight), _meta(bias)), norm, post_norm, float(res_scale))
    ref = x_out if x_out is not None else dx_out
    dev = ref.device
    dx = _like(ref)
    dy, dgate, dpw, dw, db, dscale, dshift = (
        None if t is None else _like(t) for t in (y, gate, post_weight, weight, bias, scale, shift))
    ws = None
    if dgate is not None or dscale is not None or dshift is not None or dpw is not None or dw is not None \
            or db is not None:
        ws = _workspace(dev, _size(dev, "basa_gated_norm_bwd_workspace_size", plan), workspace)
    _on(dev, _lib.load().basa_gated_norm_bwd, "basa_gated_norm_bwd", _p(dh), _p(x_out) if norm is not None else None,
        _p(stats) if plan.use_stats else None, _p(y) if plan.use_y else None, _p(dx_out), _p(gate), _p(post_weight),
        _p(weight), _p(bias), _p(scale), dx.data_ptr(), _p(dy), _p(dgate), _p(dpw), _p(dw), _p(db), _p(dscale),
        _p(dshift), _p(ws), plan.params)
    return GatedNormGrads(dx, dy, dgate, dpw, dw, db, dscale, dshift)
