"""Refusals of the calls around the attention (qkv_rope, gated_norm and their
backwards), on the host: every argument error is found before a launch, so none
of these need a GPU.  Device pointers are made-up addresses that are never used."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_diffusion_basa_b200 import build
    build.build()
    from sparse_attention_diffusion_basa_b200 import _lib
    return _lib.load()


A = 0x10000  # a 16-byte aligned address


def rope(**kw):
    from sparse_attention_diffusion_basa_b200._lib import BasaRopeParams
    p = BasaRopeParams(1, 4, 2, 1, 8, 8, 64, 0, 32, 32, 0, 1, 1e-6, 1, 1, 1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_rope(lib, p, **kw):
    a = dict(q=A, k=A, v=A, qw=A, kw=A, table=A, qo=A, ko=A, vo=A)
    a.update(kw)
    return lib.basa_qkv_rope(*a.values(), ctypes.byref(p) if p else None, None)


def call_rope_bwd(lib, p, **kw):
    a = dict(gq=A, gk=A, gv=A, q=A, k=A, qw=A, kw=A, table=A, dq=A, dk=A, dv=A, dqw=A, dkw=A, ws=A)
    a.update(kw)
    return lib.basa_qkv_rope_bwd(*a.values(), ctypes.byref(p) if p else None, None)


BAD_ROPE = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-4), INVALID), (dict(Hkv=-1), INVALID),
    (dict(Hkv=3), INVALID), (dict(d=0), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(ah=31), INVALID), (dict(at=-2), INVALID), (dict(aw=34), INVALID), (dict(layout=2), INVALID),
    (dict(layout=1, aw=24), UNSUPPORTED), (dict(norm=3), INVALID), (dict(norm=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(out_dtype=0), UNSUPPORTED),
    (dict(out_dtype=9), INVALID), (dict(w_dtype=2), INVALID), (dict(q_descale=-1.0), INVALID),
    (dict(v_descale=float("inf")), INVALID), (dict(k_descale=float("nan")), INVALID),
    (dict(ldq=128), INVALID), (dict(ldq=260), ALIGN), (dict(ldv=-8), INVALID), (dict(ldk=1 << 40), UNSUPPORTED),
    (dict(norm=2, H=512, Hkv=512), UNSUPPORTED), (dict(H=32768, Hkv=1), UNSUPPORTED),
    (dict(B=1 << 16, T=1 << 16), UNSUPPORTED), (dict(T=1 << 30, at=64, ah=0, aw=0, Hg=1, Wg=8), UNSUPPORTED),
]


@pytest.mark.parametrize("fields,code", BAD_ROPE)
def test_rope_params_refused(lib, fields, code):
    assert call_rope(lib, rope(**fields)) == code
    assert lib.basa_rope_table_pairs(ctypes.byref(rope(**fields))) == 0
    assert lib.basa_qkv_rope_bwd_workspace_size(ctypes.byref(rope(**fields))) == 0
    assert call_rope_bwd(lib, rope(**fields)) == code


def test_rope_pointers_refused(lib):
    assert call_rope(lib, None) == INVALID
    for name in ("q", "k", "qo", "ko", "vo", "v", "table"):
        assert call_rope(lib, rope(), **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "qw", "kw", "table", "qo", "ko", "vo"):
        assert call_rope(lib, rope(), **{name: A + 8}) == ALIGN, name
    assert call_rope(lib, rope(norm=0)) == INVALID            # weights without a norm
    assert call_rope_bwd(lib, None) == INVALID
    for name in ("gq", "gk", "q", "k", "dq", "dk", "dv", "gv", "table"):
        assert call_rope_bwd(lib, rope(), **{name: None}) == INVALID, name
    for name in ("gq", "gk", "gv", "q", "k", "qw", "kw", "table", "dq", "dk", "dv", "dqw", "dkw", "ws"):
        assert call_rope_bwd(lib, rope(), **{name: A + 4}) == ALIGN, name
    assert call_rope_bwd(lib, rope(), ws=None) == WORKSPACE
    assert call_rope_bwd(lib, rope(), qw=None) == INVALID     # a gradient of a weight there is not
    assert call_rope_bwd(lib, rope(out_dtype=2)) == UNSUPPORTED
    # empty problems touch nothing
    for f in (dict(B=0), dict(T=0), dict(Wg=0), dict(H=0, Hkv=0)):
        assert call_rope(lib, rope(**f), q=None) == OK
        assert call_rope_bwd(lib, rope(**f), q=None, dqw=None, dkw=None) == OK


def test_rope_table_refused(lib):
    d3 = ctypes.c_double * 3
    zero, one = d3(0, 0, 0), d3(1, 1, 1)
    f = lambda theta=1e4, s=zero, e=one, t=A, p=None: lib.basa_rope_table(  # noqa: E731
        t, theta, s, e, ctypes.byref(p or rope()), None)
    assert f(theta=0.0) == INVALID and f(theta=float("inf")) == INVALID and f(theta=float("nan")) == INVALID
    assert f(s=None) == INVALID and f(e=None) == INVALID
    assert f(s=d3(0, float("nan"), 0)) == INVALID and f(e=d3(0, 0, float("inf"))) == INVALID
    assert f(t=None) == INVALID and f(t=A + 8) == ALIGN
    assert f(p=rope(ah=0, aw=0), t=None) == OK                # nothing is rotated
    assert lib.basa_rope_table_pairs(ctypes.byref(rope(T=3, at=8, ah=32, aw=16))) == 3 * 4 + 8 * 16 + 8 * 8


def test_rope_workspace_holds_every_partial_row(lib):
    for f in (dict(), dict(norm=2), dict(B=64, Hg=128, Wg=128), dict(H=24, Hkv=8, d=128, norm=2)):
        n = lib.basa_qkv_rope_bwd_workspace_size(ctypes.byref(rope(**f)))
        assert n > 0 and n % 256 == 0
    assert lib.basa_qkv_rope_bwd_workspace_size(ctypes.byref(rope(norm=0))) == 0


def gnorm(**kw):
    from sparse_attention_diffusion_basa_b200._lib import BasaGnormParams
    p = BasaGnormParams(12, 3, 64, 1, 2, 1e-6, 1e-6, 1.0, 1, 1, 1, 1, 64, 64, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_gnorm(lib, p, **kw):
    a = dict(x=A, y=A, gate=A, pw=A, w=A, b=A, scale=A, shift=A, xo=A, h=A, stats=A)
    a.update(kw)
    return lib.basa_gated_norm(*a.values(), ctypes.byref(p) if p else None, None)


def call_gnorm_bwd(lib, p, **kw):
    a = dict(gh=A, xo=A, stats=A, y=A, gx=A, gate=A, pw=A, w=A, b=A, scale=A, dx=A, dy=A, dgate=A, dpw=A, dw=A,
             db=A, dscale=A, dshift=A, ws=A)
    a.update(kw)
    return lib.basa_gated_norm_bwd(*a.values(), ctypes.byref(p) if p else None, None)


BAD_GNORM = [
    (dict(rows=-1), INVALID), (dict(groups=0), INVALID), (dict(groups=5), SHAPE), (dict(C=0), INVALID),
    (dict(C=60), UNSUPPORTED), (dict(C=8200), UNSUPPORTED), (dict(norm=3), INVALID), (dict(post_norm=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(post_eps=-1.0), INVALID),
    (dict(post_eps=float("inf")), INVALID), (dict(res_scale=float("nan")), INVALID),
    (dict(res_scale=float("inf")), INVALID), (dict(x_dtype=2), UNSUPPORTED), (dict(dtype=7), INVALID),
    (dict(dtype=0), UNSUPPORTED), (dict(mod_dtype=2), UNSUPPORTED), (dict(w_dtype=-1), INVALID),
    (dict(ld_gate=-8), INVALID), (dict(ld_scale=60), ALIGN), (dict(ld_shift=1 << 40), UNSUPPORTED),
    (dict(rows=3 << 40), UNSUPPORTED),
]


@pytest.mark.parametrize("fields,code", BAD_GNORM)
def test_gnorm_params_refused(lib, fields, code):
    assert call_gnorm(lib, gnorm(**fields)) == code
    assert call_gnorm_bwd(lib, gnorm(**fields)) == code
    assert lib.basa_gated_norm_bwd_workspace_size(ctypes.byref(gnorm(**fields))) == 0


def test_gnorm_pointers_refused(lib):
    assert call_gnorm(lib, None) == INVALID and call_gnorm_bwd(lib, None) == INVALID
    for name in ("x", "xo", "h", "y"):                        # y: its gate and post-norm are left alone
        assert call_gnorm(lib, gnorm(), **{name: None}) == INVALID, name
    for name in ("x", "y", "gate", "pw", "w", "b", "scale", "shift", "xo", "h", "stats"):
        assert call_gnorm(lib, gnorm(), **{name: A + 8}) == ALIGN, name
    assert call_gnorm(lib, gnorm(norm=0)) == INVALID          # h without a norm
    assert call_gnorm(lib, gnorm(norm=0), h=None, w=None, b=None, scale=None) == INVALID  # shift
    assert call_gnorm(lib, gnorm(post_norm=0)) == INVALID     # post_weight without a post-norm
    none = dict(y=None, gate=None, pw=None, xo=None)
    assert call_gnorm(lib, gnorm(post_norm=0), **{**none, "gate": A}) == INVALID
    assert call_gnorm(lib, gnorm(post_norm=0), **{**none, "xo": A}) == INVALID
    assert call_gnorm(lib, gnorm(), **none) == INVALID        # a post-norm of nothing
    assert call_gnorm(lib, gnorm(rows=0), x=None) == OK
    for name in ("gh", "xo", "stats", "y", "dx", "dy", "gate", "pw", "w", "b", "scale"):
        assert call_gnorm_bwd(lib, gnorm(), **{name: None}) == INVALID, name
    for name in ("gh", "xo", "stats", "y", "gx", "gate", "pw", "w", "b", "scale", "dx", "dy", "dgate", "dpw", "dw",
                 "db", "dscale", "dshift", "ws"):
        assert call_gnorm_bwd(lib, gnorm(), **{name: A + 2}) == ALIGN, name
    assert call_gnorm_bwd(lib, gnorm(), ws=None) == WORKSPACE
    lone = dict(gh=None, w=None, b=None, scale=None, dw=None, db=None, dscale=None, dshift=None)
    assert call_gnorm_bwd(lib, gnorm(norm=0), **{**lone, "gx": None}) == INVALID  # no gradient comes in
    assert call_gnorm_bwd(lib, gnorm(norm=0), **{**lone, "dshift": A}) == INVALID
    assert call_gnorm_bwd(lib, gnorm(post_norm=0)) == INVALID


def test_python_refusals():
    import sparse_attention_diffusion_basa_b200 as basa
    q = torch.zeros(1, 1, 4, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        basa.qkv_rope(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        basa.qkv_rope_bwd(q, q, None, q, q)
    with pytest.raises(TypeError):
        basa.qkv_rope(None, q)
    x = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        basa.gated_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        basa.gated_norm_bwd(x, x, x)
    with pytest.raises(TypeError):
        basa.gated_norm("x")
    with pytest.raises(ValueError, match="CUDA"):
        basa.rope_table((1, 4, 4), (0, 32, 32), device="cpu")


def test_row_strides():
    from sparse_attention_diffusion_basa_b200.block import _row_stride
    f = lambda t, n: _row_stride(t.shape, t.stride(), n, "t")  # noqa: E731
    t = torch.zeros(2, 3, 4, 5, 7, 16)
    assert f(t, 4) == 7 * 16
    assert f(t[..., :2, :], 4) == 7 * 16
    assert f(t[:, :, :, ::2], 3) == 5 * 7 * 16      # the fourth dim is not walked
    assert f(torch.zeros(1, 1, 1, 1, 7, 16), 4) is None
    assert f(torch.zeros(3, 16)[:, :8].expand(3, 8), 1) == 16
    assert f(torch.zeros(16).expand(3, 16), 1) == 0
    for bad in (t[:, :, :, ::2], t[:, :2], t.transpose(1, 2)):
        with pytest.raises(ValueError, match="one stride"):
            f(bad, 4)
