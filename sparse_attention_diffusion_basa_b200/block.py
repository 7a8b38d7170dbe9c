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
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import (BASA_BF16, BASA_F32, BASA_FP8_E4M3, BASA_NORM, BASA_ROPE_LAYOUT, BASA_ROPE_NORM,
                   BasaGnormParams, BasaRopeParams)

_DT = {torch.float32: BASA_F32, torch.bfloat16: BASA_BF16, torch.float8_e4m3fn: BASA_FP8_E4M3}


def _code(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {key!r}") from None


def _on(t: torch.Tensor, fn, what: str, *args):
    """Calls ``fn`` with t's device current and its stream as the last argument."""
    dev = t.device
    if torch.cuda.current_device() == dev.index:
        _lib.check(fn(*args, torch.cuda.current_stream(dev).cuda_stream), what)
    else:
        with torch.cuda.device(dev):
            _lib.check(fn(*args, torch.cuda.current_stream(dev).cuda_stream), what)


def _size(t: torch.Tensor, fn, prm) -> int:
    """Workspace bytes, asked with t's device current (they go by its SMs)."""
    if torch.cuda.current_device() == t.device.index:
        return int(fn(ctypes.byref(prm)))
    with torch.cuda.device(t.device):
        return int(fn(ctypes.byref(prm)))


def _workspace(t, need, workspace):
    if not need:
        return None
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=t.device)
    if workspace.device != t.device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} contiguous bytes on {t.device}")
    return workspace


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _tensor(t, ref, name, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if ref is not None and t.device != ref.device:
        raise ValueError(f"{name} must be on {ref.device}, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")


_FLOAT = (torch.float32, torch.bfloat16)


def _row_stride(shape, stride, n, name) -> int:
    """Elements between consecutive rows when the first n dims are walked in order."""
    ld = expect = None
    for size, st in zip(reversed(shape[:n]), reversed(stride[:n])):
        if size == 1:
            continue
        if ld is None:
            ld = st
        elif st != expect:
            raise ValueError(f"the rows of {name} {tuple(shape)} must lie at one stride, got {tuple(stride)}")
        expect = st * size
    return ld


# ---------------------------------------------------------------------------
# q/k/v preparation
# ---------------------------------------------------------------------------
def _heads(t, ref, name, dtypes, dense=False) -> int:
    """Checks a [B, T, Hg, Wg, heads, d] (or text [B, L, heads, d]) tensor; its row stride, 0 = dense."""
    _tensor(t, ref, name, dtypes)
    if t.dim() not in (4, 6):
        raise ValueError(f"{name} must be [B, T, Hg, Wg, heads, d] or [B, L, heads, d], got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    if dense:
        raise ValueError(f"{name} must be contiguous")
    shape, stride = t.shape, t.stride()
    if t.numel() == 0:
        return 0
    if (shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1]):
        raise ValueError(f"the heads of {name} must be dense, got strides {tuple(stride)}")
    ld = _row_stride(shape, stride, t.dim() - 2, name)
    if ld is None:
        return 0
    if ld < shape[-1] * shape[-2]:
        raise ValueError(f"the rows of {name} overlap: strides {tuple(stride)}")
    return ld


def _rope_params(q, k, axes, layout, norm, eps, out_dtype, descale, lds, w_dtype) -> BasaRopeParams:
    if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"k {tuple(k.shape)} must match q {tuple(q.shape)} except in heads")
    H, Hkv = q.shape[-2], k.shape[-2]
    if H != Hkv and (Hkv == 0 or H % Hkv):
        raise ValueError(f"q heads {H} must be a multiple of k/v heads {Hkv}")
    B = q.shape[0]
    T, Hg, Wg = q.shape[1:4] if q.dim() == 6 else (1, 1, q.shape[1])
    at, ah, aw = (int(a) for a in axes)
    return BasaRopeParams(B, H, Hkv, T, Hg, Wg, q.shape[-1], at, ah, aw, _code(BASA_ROPE_LAYOUT, layout, "layout"),
                          _code(BASA_ROPE_NORM, norm, "norm"), float(eps), _DT[q.dtype], _DT[out_dtype],
                          _DT[w_dtype], *(float(x) for x in descale), *lds)


def _pairs(prm) -> int:
    return prm.T * (prm.at // 2) + prm.Hg * (prm.ah // 2) + prm.Wg * (prm.aw // 2)


def _check_table(table, q, prm):
    n = _pairs(prm)
    if n == 0:
        return None
    _tensor(table, q, "table", (torch.float32,))
    if table.numel() != 2 * n or not table.is_contiguous():
        raise ValueError(f"table must hold {n} contiguous (cos, sin) pairs for this grid and these axes, "
                         f"got {tuple(table.shape)}")
    return table


def _weights(q, k, q_weight, k_weight, norm):
    """Checks the norm weights; their dtype."""
    dtype = None
    for w, t, name in ((q_weight, q, "q_weight"), (k_weight, k, "k_weight")):
        if w is None:
            continue
        if norm is None:
            raise ValueError(f"{name} needs a norm")
        _tensor(w, q, name, _FLOAT)
        n = t.shape[-1] * (t.shape[-2] if norm == "token" else 1)
        if w.numel() != n or not w.is_contiguous():
            raise ValueError(f"{name} must be {n} contiguous values, got {tuple(w.shape)}")
        if dtype not in (None, w.dtype):
            raise TypeError("q_weight and k_weight must share a dtype")
        dtype = w.dtype
    return dtype or torch.float32


def rope_table(grid, axes, theta: float = 10000.0, start=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0),
               device=None, out=None, stream=None) -> torch.Tensor:
    """The (cos, sin) pairs of a grid (T, Hg, Wg) for ``axes`` = rotated elements of a
    head per axis -> fp32 [T*at/2 + Hg*ah/2 + Wg*aw/2, 2].

    Coordinate i of an axis stands at position start + step * i; pair j turns by
    position * theta^(-2j / width).  Keep it while grid and positions stay."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rope_table(grid, axes, theta, start, step, device, out)
    T, Hg, Wg = (int(g) for g in grid)
    at, ah, aw = (int(a) for a in axes)
    d = 32
    while d < at + ah + aw and d < 128:
        d *= 2
    prm = BasaRopeParams(1, 1, 1, T, Hg, Wg, d, at, ah, aw, 0, 0, 1.0, BASA_F32, BASA_F32, BASA_F32)
    lib = _lib.load()
    pos = [(ctypes.c_double * 3)(*(float(x) for x in v)) for v in (start, step)]
    if out is None:
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("device must be a CUDA device")
        out = torch.empty((max(_pairs(prm), 0), 2), dtype=torch.float32, device=dev)
    else:
        _check_table(out, out, prm)
    _on(out, lib.basa_rope_table, "basa_rope_table", _p(out), float(theta), *pos, ctypes.byref(prm))
    return out


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
    output may be its own dense input."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qkv_rope(q, k, v, table, axes, layout=layout, norm=norm, q_weight=q_weight, k_weight=k_weight,
                            eps=eps, out_dtype=out_dtype, descale=descale, out=out)
    lds = [_heads(q, None, "q", _FLOAT), _heads(k, q, "k", (q.dtype,)), 0]
    if v is not None:
        lds[2] = _heads(v, q, "v", (q.dtype,))
        if v.shape != k.shape:
            raise ValueError("k and v must have the same shape")
    dt = q.dtype if out_dtype is None else out_dtype
    if dt not in (q.dtype, torch.float8_e4m3fn):
        raise TypeError(f"out_dtype must be {q.dtype} or torch.float8_e4m3fn, got {dt}")
    w_dtype = _weights(q, k, q_weight, k_weight, norm)
    prm = _rope_params(q, k, axes, layout, norm, eps, dt, descale, lds, w_dtype)
    table = _check_table(table, q, prm)
    if out is None:
        qo, ko = torch.empty(q.shape, dtype=dt, device=q.device), torch.empty(k.shape, dtype=dt, device=q.device)
        vo = None if v is None else torch.empty(k.shape, dtype=dt, device=q.device)
    else:
        qo, ko, vo = out
        for o, t, name in ((qo, q, "q"), (ko, k, "k"), (vo, v, "v")):
            if (o is None) != (t is None):
                raise ValueError(f"out must give {name}'s output exactly when {name} is given")
            if o is not None:
                _heads(o, q, f"{name}'s output", (dt,), dense=True)
                if o.shape != t.shape:
                    raise ValueError(f"{name}'s output must have shape {tuple(t.shape)}")
    _on(q, _lib.load().basa_qkv_rope, "basa_qkv_rope", _p(q), _p(k), _p(v), _p(q_weight), _p(k_weight), _p(table),
        _p(qo), _p(ko), _p(vo), ctypes.byref(prm))
    return qo, ko, vo


def qkv_rope_bwd(dq_out, dk_out, dv_out, q, k, table=None, axes=(0, 0, 0), *, layout="pairs", norm=None,
                 q_weight=None, k_weight=None, eps=1e-6, out=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dq_weight, dk_weight) of qkv_rope; None for what the call had not.

    ``dq_out``, ``dk_out``, ``dv_out`` (or None) are the dense gradients of its
    outputs, q and k its inputs.  ``out`` = (dq, dk, dv) gives the tensors to
    write, which may be slices of one buffer."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qkv_rope_bwd(dq_out, dk_out, dv_out, q, k, table, axes, layout=layout, norm=norm,
                                q_weight=q_weight, k_weight=k_weight, eps=eps, out=out, workspace=workspace)
    _heads(dq_out, None, "dq_out", _FLOAT, dense=True)
    _heads(dk_out, dq_out, "dk_out", (dq_out.dtype,), dense=True)
    lds = [0] * 6
    for i, (t, g, name) in enumerate(((q, dq_out, "q"), (k, dk_out, "k"))):
        if norm is None and t is None:
            continue
        lds[i] = _heads(t, dq_out, name, (dq_out.dtype,))
        if t.shape != g.shape:
            raise ValueError(f"{name} {tuple(t.shape)} must have the shape of its output's gradient {tuple(g.shape)}")
    if dv_out is not None:
        _heads(dv_out, dq_out, "dv_out", (dq_out.dtype,), dense=True)
        if dv_out.shape != dk_out.shape:
            raise ValueError("dk_out and dv_out must have the same shape")
    grads = (dq_out, dk_out, dv_out)
    if out is None:
        out = tuple(None if g is None else torch.empty_like(g) for g in grads)
    else:
        out = tuple(out)
        for i, (o, g) in enumerate(zip(out, grads)):
            if (o is None) != (g is None):
                raise ValueError("out must give dv exactly when dv_out is given")
            if o is not None:
                lds[3 + i] = _heads(o, dq_out, "a gradient", (dq_out.dtype,))
                if o.shape != g.shape:
                    raise ValueError(f"a gradient must have shape {tuple(g.shape)}, got {tuple(o.shape)}")
    w_dtype = _weights(dq_out, dk_out, q_weight, k_weight, norm)
    prm = _rope_params(dq_out, dk_out, axes, layout, norm, eps, dq_out.dtype, (0.0, 0.0, 0.0), lds, w_dtype)
    table = _check_table(table, dq_out, prm)
    lib = _lib.load()
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    if dqw is not None or dkw is not None:
        workspace = _workspace(dq_out, _size(dq_out, lib.basa_qkv_rope_bwd_workspace_size, prm), workspace)
    else:
        workspace = None
    _on(dq_out, lib.basa_qkv_rope_bwd, "basa_qkv_rope_bwd", _p(dq_out), _p(dk_out), _p(dv_out),
        _p(q) if norm is not None else None, _p(k) if norm is not None else None, _p(q_weight), _p(k_weight),
        _p(table), _p(out[0]), _p(out[1]), _p(out[2]), _p(dqw), _p(dkw), _p(workspace), ctypes.byref(prm))
    return (*out, dqw, dkw)


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


def _rows(t, ref, name, dtypes, shape=None):
    _tensor(t, ref, name, dtypes)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _modulation(m, x, name):
    """(rows of a modulation, elements from one to the next; 0: one for all)."""
    _tensor(m, x, name, _FLOAT)
    C = x.shape[-1]
    lead = m.shape[:-1]
    if m.dim() < 1 or m.shape[-1] != C or (C > 1 and m.stride(-1) != 1):
        raise ValueError(f"{name} must end in {C} dense columns, got {tuple(m.shape)}")
    n = len(lead)
    if n and tuple(lead) != tuple(x.shape[:n]) and not (
            n == 2 and x.dim() == 3 and lead[0] == x.shape[0] and lead[1] and x.shape[1] % lead[1] == 0):
        raise ValueError(f"{name} {tuple(m.shape)} must be [C], or lead with dims of x {tuple(x.shape)}")
    groups = 1
    for s in lead:
        groups *= s
    return groups, _row_stride(m.shape, m.stride(), n, name) or 0


def _gnorm_params(x, y_dtype, mods, weights, norm, post_norm, eps, post_eps, res_scale) -> BasaGnormParams:
    """mods: (gate, scale, shift); weights: (post_weight, weight, bias)."""
    C = x.shape[-1]
    groups, lds, mod_dtype, w_dtype = None, [], None, None
    for m, name in zip(mods, ("gate", "scale", "shift")):
        if m is None:
            lds.append(0)
            continue
        g, ld = _modulation(m, x, name)
        if groups not in (None, g):
            raise ValueError("gate, scale and shift must have the same leading dims (expand the shorter)")
        if mod_dtype not in (None, m.dtype):
            raise TypeError("gate, scale and shift must share a dtype")
        groups, mod_dtype = g, m.dtype
        lds.append(ld)
    for w, name in zip(weights, ("post_weight", "weight", "bias")):
        if w is None:
            continue
        _rows(w, x, name, _FLOAT)
        if w.numel() != C:
            raise ValueError(f"{name} must be {C} values, got {tuple(w.shape)}")
        if w_dtype not in (None, w.dtype):
            raise TypeError("weight, bias and post_weight must share a dtype")
        w_dtype = w.dtype
    rows = 1
    for s in x.shape[:-1]:
        rows *= s
    return BasaGnormParams(rows, max(groups or 1, 1), C, _code(BASA_NORM, norm, "norm"),
                           _code(BASA_NORM, post_norm, "post_norm"), float(eps), float(post_eps), float(res_scale),
                           _DT[x.dtype], _DT[y_dtype], _DT[mod_dtype or torch.float32],
                           _DT[w_dtype or torch.float32], *lds)


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
        with torch.cuda.stream(stream):
            return gated_norm(x, y, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                              shift=shift, norm=norm, post_norm=post_norm, eps=eps, post_eps=post_eps,
                              res_scale=res_scale, h_dtype=h_dtype, return_stats=return_stats, x_out=x_out,
                              h_out=h_out)
    _rows(x, None, "x", _FLOAT)
    if x.dim() < 2:
        raise ValueError(f"x must be [..., C], got {tuple(x.shape)}")
    if y is not None:
        _rows(y, x, "y", _FLOAT, x.shape)
        if h_dtype not in (None, y.dtype):
            raise TypeError(f"h has y's dtype {y.dtype}")
        dt = y.dtype
    else:
        if gate is not None or post_norm is not None or x_out is not None or norm is None:
            raise ValueError("without y there is no gate, post_norm or x_out, and norm must be given")
        if res_scale != 1.0:
            raise ValueError("res_scale needs y")
        dt = h_dtype or x.dtype
        if dt not in _FLOAT:
            raise TypeError(f"h_dtype must be {' or '.join(map(str, _FLOAT))}, got {dt}")
    if norm is None and h_out is not None:
        raise ValueError("h_out needs a norm")
    prm = _gnorm_params(x, dt, (gate, scale, shift), (post_weight, weight, bias), norm, post_norm, eps, post_eps,
                        res_scale)
    if x_out is not None:
        _rows(x_out, x, "x_out", (x.dtype,), x.shape)
    elif y is not None:
        x_out = torch.empty_like(x)
    if h_out is not None:
        _rows(h_out, x, "h_out", (dt,), x.shape)
    elif norm is not None:
        h_out = torch.empty(x.shape, dtype=dt, device=x.device)
    stats = torch.empty((*x.shape[:-1], 4), dtype=torch.float32, device=x.device) if return_stats else None
    _on(x, _lib.load().basa_gated_norm, "basa_gated_norm", _p(x), _p(y), _p(gate), _p(post_weight), _p(weight),
        _p(bias), _p(scale), _p(shift), _p(x_out), _p(h_out), _p(stats), ctypes.byref(prm))
    x_out = x if y is None else x_out
    return (x_out, h_out, stats) if return_stats else (x_out, h_out)


def gated_norm_bwd(dh, x_out, stats, y=None, dx_out=None, *, gate=None, post_weight=None, weight=None, bias=None,
                   scale=None, shift=None, norm="layer", post_norm=None, res_scale=1.0, workspace=None, stream=None
                   ) -> GatedNormGrads:
    """Gradients of gated_norm for the gradients ``dh`` and ``dx_out`` (or None: zero) of its outputs.

    x_out and stats are the forward's (for a call without y, x_out is x); y and
    the rest as the forward was given them (shift's values are not read).  norm
    None: dh is None and dx_out is required.  dgate, dscale, dshift have the
    modulations' leading dims, dense."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_norm_bwd(dh, x_out, stats, y, dx_out, gate=gate, post_weight=post_weight, weight=weight,
                                  bias=bias, scale=scale, shift=shift, norm=norm, post_norm=post_norm,
                                  res_scale=res_scale, workspace=workspace)
    ref = x_out if x_out is not None else dx_out
    _rows(ref, None, "x_out" if x_out is not None else "dx_out", _FLOAT)
    if ref.dim() < 2:
        raise ValueError(f"x_out must be [..., C], got {tuple(ref.shape)}")
    if (dh is None) != (norm is None):
        raise ValueError("dh goes with a norm")
    if norm is not None and x_out is None:
        raise ValueError("x_out is needed with a norm")
    if norm is None and dx_out is None:
        raise ValueError("dx_out is needed without a norm")
    if y is None and (gate is not None or post_norm is not None or norm is None):
        raise ValueError("without y there is no gate or post_norm, and norm must be given")
    if y is None and res_scale != 1.0:
        raise ValueError("res_scale needs y")
    dt = dh.dtype if dh is not None else y.dtype
    if dh is not None:
        _rows(dh, ref, "dh", _FLOAT, ref.shape)
    if y is not None:
        _rows(y, ref, "y", (dt,), ref.shape)
    if dx_out is not None:
        _rows(dx_out, ref, "dx_out", (ref.dtype,), ref.shape)
    if norm is not None or post_norm is not None:
        _rows(stats, ref, "stats", (torch.float32,), torch.Size((*ref.shape[:-1], 4)))
    prm = _gnorm_params(ref, dt, (gate, scale, shift), (post_weight, weight, bias), norm, post_norm, 1.0, 1.0,
                        res_scale)
    like = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    g = GatedNormGrads(torch.empty_like(ref), like(y), like(gate), like(post_weight), like(weight), like(bias),
                       like(scale), like(shift))
    lib = _lib.load()
    if any(t is not None for t in g[2:]):
        workspace = _workspace(ref, _size(ref, lib.basa_gated_norm_bwd_workspace_size, prm), workspace)
    else:
        workspace = None
    _on(ref, lib.basa_gated_norm_bwd, "basa_gated_norm_bwd", _p(dh), _p(x_out) if norm is not None else None,
        _p(stats) if norm is not None or post_norm is not None else None,
        _p(y) if gate is not None or post_norm is not None else None, _p(dx_out), _p(gate), _p(post_weight),
        _p(weight), _p(bias), _p(scale), *(_p(t) for t in g), _p(workspace), ctypes.byref(prm))
    return g
