"""What the binding of the calls around the attention (qkv_rope, gated_norm and their backwards)
makes of its arguments, on the host: tensors are stood in for by their shapes and made-up addresses,
and the library's entry by a function that records the parameter struct, so nothing is launched."""
import ctypes
import gc
import types
import weakref

import pytest
import torch

from sparse_attention_diffusion_basa_b200 import block

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SIZE = {BF: 2, F32: 4, E4: 1}


class Stub:
    """A CUDA tensor as far as the binding looks at one."""
    _next = 1 << 32

    def __init__(self, *shape, dtype=BF, stride=None, at=None, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self._stride = tuple(torch.empty(shape, device="meta").stride()) if stride is None else stride
        if at is None:
            at = Stub._next
            Stub._next += 1 << 32
        self._at = at

    def stride(self):
        return self._stride

    def data_ptr(self):
        return self._at


@pytest.fixture
def calls(monkeypatch):
    """The parameter structs of the calls that reach the library, copied as they were then."""
    from sparse_attention_diffusion_basa_b200 import build
    build.build()
    seen = []

    def on(device, fn, what, *args):
        p = args[-1]._obj
        seen.append(type(p).from_buffer_copy(bytes(p)))
    monkeypatch.setattr(block, "_on", on)
    monkeypatch.setattr(block, "_like", lambda t, dtype=None: Stub(*t.shape, dtype=dtype or t.dtype))
    return seen


def same32(got, value):
    return got == ctypes.c_float(value).value


def test_scalar_tensors_are_read_at_every_call(calls):
    """A 0-dim tensor that is changed in place between two calls: the second call takes its new value."""
    q, k, v = Stub(1, 1, 4, 4, 2, 64), Stub(1, 1, 4, 4, 2, 64), Stub(1, 1, 4, 4, 2, 64)
    x, y = Stub(1, 6, 64), Stub(1, 6, 64)
    st = Stub(1, 6, 4, dtype=F32)
    cases = [
        (("q_descale",), lambda s: block.qkv_rope(q, k, v, out_dtype=E4, descale=(s, 1.0, 1.0))),
        (("k_descale", "v_descale"), lambda s: block.qkv_rope(q, k, v, out_dtype=E4, descale=[1.0, s, s])),
        (("eps",), lambda s: block.qkv_rope(q, k, v, norm="head", eps=s)),
        (("eps",), lambda s: block.qkv_rope_bwd(q, k, v, q, k, norm="head", eps=s)),
        (("eps",), lambda s: block.gated_norm(x, y, eps=s)),
        (("post_eps",), lambda s: block.gated_norm(x, y, post_norm="rms", post_eps=s)),
        (("res_scale",), lambda s: block.gated_norm(x, y, res_scale=s)),
        (("res_scale",), lambda s: block.gated_norm_bwd(x, x, st, y, res_scale=s)),
    ]
    for fields, call in cases:
        s = torch.tensor(0.25)
        for value in (0.25, 0.5, 0.125):
            s.fill_(value)
            call(s)
            assert all(same32(getattr(calls[-1], f), value) for f in fields), (fields, value)


def test_whole_number_tensors_are_read_at_every_call(calls):
    n, m = torch.tensor(16), torch.tensor(48)
    q, table = Stub(1, 1, 4, 4, 2, 64), Stub(4 * 32, 2, dtype=F32)
    for rows, columns in ((16, 48), (48, 16), (32, 32)):
        n.fill_(rows)
        m.fill_(columns)
        block.qkv_rope(q, q, None, table, (0, n, m))
        assert (calls[-1].ah, calls[-1].aw) == (rows, columns)
        block.qkv_rope_bwd(q, q, None, None, None, table, (0, n, m))
        assert (calls[-1].ah, calls[-1].aw) == (rows, columns)
        block.rope_table((1, n, m), (0, 8, 8), out=Stub(4 * 64, 2, dtype=F32))
        assert (calls[-1].Hg, calls[-1].Wg) == (rows, columns)


def test_no_scalar_tensor_is_kept(calls):
    q, x = Stub(1, 1, 4, 4, 2, 64), Stub(1, 6, 64)
    s = torch.tensor(0.5)
    kept = weakref.ref(s)
    block.qkv_rope(q, q, q, out_dtype=E4, norm="head", descale=(s, s, s), eps=s)
    block.gated_norm(x, x, eps=s, post_eps=s, res_scale=s)
    del s
    gc.collect()
    assert kept() is None


def test_factors_without_a_reciprocal_are_refused():
    """An e4m3 factor whose reciprocal leaves fp32's normal numbers: zeros would become NaN."""
    from sparse_attention_diffusion_basa_b200 import _lib, build
    build.build()
    lib, at16 = _lib.load(), 0x10000  # an address that is never used
    for factor, code in ((1e-45, 1), (1e-39, 1), (7e-31, 1), (1.5e30, 1), (3e38, 1), (8e-31, 4), (1.2e30, 4)):
        for name in ("q_descale", "k_descale", "v_descale"):
            p = _lib.BasaRopeParams(1, 2, 2, 1, 8, 8, 64, 0, 0, 0, 0, 0, 1e-6, 1, 2, 1)
            setattr(p, name, factor)
            # an unaligned output is found behind the parameters, and ahead of a launch
            got = lib.basa_qkv_rope(at16, at16, at16, None, None, None, at16, at16, at16 + 8, ctypes.byref(p), None)
            assert got == code, (name, factor)
            p.out_dtype = 1  # the factors of a bf16 output are not looked at
            got = lib.basa_qkv_rope(at16, at16, at16, None, None, None, at16, at16, at16 + 8, ctypes.byref(p), None)
            assert got == 4, (name, factor)


def test_modulations_of_unlike_lengths_follow_the_advice(calls):
    """gate a sample, scale and shift a frame: what the refusal asks for is then accepted."""
    x = Stub(2, 6, 64)
    gate, scale = Stub(2, 64), Stub(2, 3, 64)
    with pytest.raises(ValueError, match="leading dims") as e:
        block.gated_norm(x, x, gate=gate, scale=scale)
    assert "contiguous" in str(e.value)
    block.gated_norm(x, x, gate=Stub(2, 3, 64), scale=scale)
    assert calls[-1].groups == 6 and calls[-1].ld_gate == 64
    block.gated_norm(x, x, gate=Stub(2, 64, stride=(0, 1)), scale=Stub(2, 64))  # one row for all samples
    assert calls[-1].groups == 2 and calls[-1].ld_gate == 0
    with pytest.raises(ValueError, match="contiguous"):  # expanded, but rows at two strides
        block.gated_norm(x, x, gate=Stub(2, 3, 64, stride=(64, 0, 1)), scale=scale)


def test_stream_of_another_device_is_refused(calls):
    """The tensors lie on cuda:0, the stream on cuda:1: the call could not run on that stream."""
    far = types.SimpleNamespace(device=torch.device("cuda", 1))
    q, x, st = Stub(1, 1, 4, 4, 2, 64), Stub(1, 6, 64), Stub(1, 6, 4, dtype=F32)
    for call in (lambda: block.qkv_rope(q, q, q, stream=far),
                 lambda: block.qkv_rope_bwd(q, q, q, q, q, stream=far),
                 lambda: block.gated_norm(x, x, stream=far),
                 lambda: block.gated_norm_bwd(x, x, st, x, stream=far),
                 lambda: block.gated_norm_bwd(None, None, None, x, x, norm=None, stream=far),
                 lambda: block.rope_table((1, 4, 4), (0, 8, 8), out=Stub(32, 2, dtype=F32), stream=far),
                 lambda: block.rope_table((1, 4, 4), (0, 8, 8), device="cuda:0", stream=far)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not calls


@pytest.fixture
def codes(calls, monkeypatch):
    """The library's own answers to calls on made-up addresses, which it must give ahead of a launch:
    without a device, a call that passes every check ends in BASA_ERR_CUDA."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses are for a machine without a device")
    seen = []

    def on(device, fn, what, *args):
        seen.append(fn(*args, None))
    monkeypatch.setattr(block, "_on", on)
    return seen


PASSED, REFUSED = 6, 1


def at(t, byte, **kw):
    shape = kw.get("shape", t.shape)
    return Stub(*shape, dtype=kw.get("dtype", t.dtype), stride=kw.get("stride"), at=t.data_ptr() + byte)


def test_overlapping_outputs_are_refused(codes):
    q, k, v = (Stub(1, 1, 4, 4, 2, 64) for _ in range(3))
    nbytes = 16 * 2 * 64 * 2
    new = lambda dtype=BF: Stub(*q.shape, dtype=dtype)  # noqa: E731
    t, table, w = new(), Stub(4 * 32, 2, dtype=F32), Stub(64)
    axes = (0, 32, 32)
    f = lambda out, **kw: block.qkv_rope(q, k, v, table, axes, norm="head", q_weight=w, out=out, **kw)  # noqa: E731
    for out in ((new(), new(), new()), (q, k, v), (t, at(t, nbytes), at(t, 2 * nbytes)), (q, new(), new())):
        f(out)
        assert codes[-1] == PASSED
    for out in ((t, t, new()), (t, new(), t), (new(), t, t), (t, at(t, nbytes - 16), v), (k, q, v), (k, new(), v),
                (at(q, 16), k, v), (at(q, -16), k, v), (t, v, new()), (at(w, 128 - nbytes, shape=q.shape), k, v),
                (at(table, 16, shape=q.shape, dtype=BF), k, v)):
        f(out)
        assert codes[-1] == REFUSED
    # in place only where a token's bytes stay where they are
    f((new(E4), new(E4), new(E4)), out_dtype=E4)
    assert codes[-1] == PASSED
    f((at(q, 0, dtype=E4), new(E4), new(E4)), out_dtype=E4)
    assert codes[-1] == REFUSED
    # the same tensor as both inputs: neither output can take its place
    block.qkv_rope(q, q, None, table, axes, out=(new(), new(), None))
    assert codes[-1] == PASSED
    block.qkv_rope(q, q, None, table, axes, out=(q, new(), None))
    assert codes[-1] == REFUSED
    # slices of one projection: dense outputs may not lie in it, one in a gap between its rows may
    rows = (16 * 512, 16 * 512, 4 * 512, 512, 64, 1)
    whole = Stub(*q.shape, stride=rows)
    x = [at(whole, 256 * i, stride=rows) for i in range(3)]
    one = Stub(1, 1, 1, 1, 2, 64)
    block.qkv_rope(*x, table, axes, out=(new(), new(), new()))
    assert codes[-1] == PASSED
    block.qkv_rope(*x, table, axes, out=(at(whole, 0), new(), new()))
    assert codes[-1] == REFUSED
    block.qkv_rope(x[0], x[1], None, table, axes, out=(at(whole, 768, shape=q.shape), new(), None))
    assert codes[-1] == REFUSED
    block.qkv_rope(one, one, None, out=(at(whole, 768, shape=one.shape), at(whole, 1792, shape=one.shape), None))
    assert codes[-1] == PASSED


def test_overlapping_gradients_are_refused(codes):
    shape = (1, 1, 4, 4, 2, 64)
    q, k, gq, gk, gv = (Stub(*shape) for _ in range(5))
    table, axes = Stub(4 * 32, 2, dtype=F32), (0, 32, 32)

    def sliced(ld, *offs):
        whole = Stub(*shape, stride=(16 * ld, 16 * ld, 4 * ld, ld, 64, 1))
        return [at(whole, 2 * o, stride=whole.stride()) for o in offs]
    f = lambda out, **kw: block.qkv_rope_bwd(gq, gk, gv, q, k, table, axes, norm="head", out=out, **kw)  # noqa: E731
    for out in (sliced(384, 0, 128, 256), sliced(400, 8, 136, 264), sliced(384, 256, 0, 128),
                sliced(512, 384 + 512 * 16, 128, 256), sliced(384, 0, 384 + 128, 768 + 256), (gq, gk, gv)):
        f(out)
        assert codes[-1] == PASSED
    for out in (sliced(384, 0, 120, 256), sliced(384, 0, 128, 128), sliced(384, 0, 128, 264), (gk, gq, gv),
                (gq, gq, gv), (q, gk, gv), (Stub(*shape), k, gv), sliced(384, 128, 0, 384 + 8)):
        f(out)
        assert codes[-1] == REFUSED
    # without a norm q and k are not read
    block.qkv_rope_bwd(gq, gk, gv, q, k, table, axes, out=(q, k, gv))
    assert codes[-1] == PASSED
    # rows at different strides that never meet, and that do
    a = Stub(*shape, stride=(16 * 256, 16 * 256, 4 * 256, 256, 64, 1))
    wide = (16 * 512, 16 * 512, 4 * 512, 512, 64, 1)
    f((a, at(a, 2 * 128, stride=wide), Stub(*shape)))
    assert codes[-1] == PASSED
    f((a, at(a, 2 * 136, stride=wide), Stub(*shape)))
    assert codes[-1] == REFUSED


def test_overlapping_border_outputs_are_refused(codes):
    x, y = Stub(2, 6, 64), Stub(2, 6, 64)
    gate, w, t = Stub(2, 64), Stub(64), Stub(2, 6, 64)
    nbytes = 2 * 6 * 64 * 2
    f = lambda **kw: block.gated_norm(x, y, gate=gate, weight=w, **kw)  # noqa: E731
    for kw in (dict(x_out=x, h_out=y), dict(x_out=x), dict(h_out=y), dict(x_out=t, h_out=at(t, nbytes))):
        f(**kw)
        assert codes[-1] == PASSED
    for kw in (dict(x_out=t, h_out=t), dict(x_out=y), dict(h_out=x), dict(x_out=y, h_out=x), dict(x_out=x, h_out=x),
               dict(x_out=t, h_out=at(t, nbytes - 16)), dict(x_out=at(x, 16)), dict(h_out=at(y, -16)),
               dict(h_out=at(gate, 0, shape=x.shape)), dict(h_out=at(gate, 128 - nbytes + 16, shape=x.shape)),
               dict(x_out=at(w, 16 - nbytes, shape=x.shape))):
        f(**kw)
        assert codes[-1] == REFUSED
    block.gated_norm(x, x, x_out=x)  # the same tensor joins itself: the sum has no place of its own
    assert codes[-1] == REFUSED
    block.gated_norm(x, None, h_out=t)
    assert codes[-1] == PASSED
    block.gated_norm(x, None, h_out=x)
    assert codes[-1] == REFUSED


def test_overlapping_border_gradients_are_refused(codes):
    """The C entry, which takes every output from its caller."""
    from sparse_attention_diffusion_basa_b200 import _lib
    prm = _lib.BasaGnormParams(12, 3, 64, 1, 2, 1e-6, 1e-6, 1.0, 1, 1, 1, 1, 64, 64, 64)
    ins = ["gh", "xo", "stats", "y", "gx", "gate", "pw", "w", "b", "scale"]
    outs = ["dx", "dy", "dgate", "dpw", "dw", "db", "dscale", "dshift", "ws"]
    base = {name: (i + 1) << 32 for i, name in enumerate(ins + outs)}

    def call(**kw):
        return _lib.load().basa_gated_norm_bwd(*{**base, **kw}.values(), ctypes.byref(prm), None)
    assert call() == PASSED and call(dx=base["gx"]) == PASSED
    for i, name in enumerate(outs):
        for other in ins + outs[:i]:
            if (name, other) != ("dx", "gx"):
                assert call(**{name: base[other]}) == REFUSED, (name, other)
    assert call(dgate=base["dscale"] + 3 * 64 * 2) == PASSED
    assert call(dgate=base["dscale"] + 3 * 64 * 2 - 16) == REFUSED
    need = _lib.load().basa_gated_norm_bwd_workspace_size(ctypes.byref(prm))
    assert call(dw=base["ws"] + need) == PASSED and call(dw=base["ws"] + need - 256) == REFUSED


def test_positions_and_factors_come_in_threes(calls):
    """start and step give one value an axis, descale one of q, k, v; a missing one is not taken for
    zero (or for a row stride, which lies behind the factors in the struct)."""
    out = Stub(32, 2, dtype=F32)
    block.rope_table((1, 4, 4), (0, 8, 8), start=(0, 1, 2), step=[1, 1, 0.5], out=out)
    assert len(calls) == 1
    for kw in (dict(start=(1.0, 2.0)), dict(step=(1.0, 1.0)), dict(start=()), dict(step=(1.0,) * 4)):
        with pytest.raises(ValueError, match="three"):
            block.rope_table((1, 4, 4), (0, 8, 8), out=out, **kw)
    assert len(calls) == 1
    q = Stub(1, 1, 4, 4, 2, 64)
    for descale in ((0.5,), (0.5, 0.5), (0.5,) * 4):
        with pytest.raises(ValueError, match="three"):
            block.qkv_rope(q, q, q, out_dtype=E4, descale=descale)
    assert len(calls) == 1


def test_no_query_heads_beside_key_heads_is_refused():
    """Zero query heads with K/V heads: a call that would leave k's and v's outputs unwritten."""
    from sparse_attention_diffusion_basa_b200 import _lib, build
    build.build()
    lib, at16 = _lib.load(), 0x10000  # an address that is never used
    for norm in (0, 1, 2):
        p = _lib.BasaRopeParams(1, 0, 2, 1, 8, 8, 64, 0, 32, 32, 0, norm, 1e-6, 1, 1, 1)
        w = at16 if norm else None
        args = [at16] * 3 + [w, w] + [at16] * 4
        assert lib.basa_qkv_rope(*args, ctypes.byref(p), None) == 1
        args = [at16] * 5 + [w, w] + [at16] * 4 + [w, w, at16]
        assert lib.basa_qkv_rope_bwd(*args, ctypes.byref(p), None) == 1
    q, k = Stub(1, 1, 8, 8, 0, 64), Stub(1, 1, 8, 8, 2, 64)
    with pytest.raises(ValueError, match="heads"):
        block.qkv_rope(q, k, k)
    with pytest.raises(ValueError, match="heads"):
        block.qkv_rope_bwd(q, k, k, q, k)


def test_no_tokens_with_a_modulation_each(calls, monkeypatch):
    """An empty batch's modulations, one for each of its tokens: an empty call, as with one a sample."""
    monkeypatch.setattr(block, "_size", lambda *a: 0)
    for lead in ((2, 0), (0, 3), (0, 0)):
        x, st = Stub(*lead, 64), Stub(*lead, 4, dtype=F32)
        m = Stub(*lead, 64)
        block.gated_norm(x, x, gate=m, scale=m, shift=m)
        assert calls[-1].rows == 0
        block.gated_norm_bwd(x, x, st, x, gate=m, scale=m, shift=m)
        assert calls[-1].rows == 0


def test_workspaces_grow_with_what_they_hold():
    """At least one partial row of fp32 sums of each kind, and with more tokens or columns more; whole
    steps of 256 bytes.  (That a call keeps to the size is for a device to show.)"""
    from sparse_attention_diffusion_basa_b200 import _lib, build
    build.build()
    lib = _lib.load()

    def rope(norm, H, Hkv, d, tokens):
        p = _lib.BasaRopeParams(1, H, Hkv, 1, 1, tokens, d, 0, 0, 0, 0, norm, 1e-6, 1, 1, 1)
        n = lib.basa_qkv_rope_bwd_workspace_size(ctypes.byref(p))
        # one row at least of q's and of k's weights
        assert n % 256 == 0 and n >= 4 * d * (H + Hkv if norm == 2 else 2), (norm, H, Hkv, d, tokens, n)
        return n

    def border(rows, groups, C):
        p = _lib.BasaGnormParams(rows, groups, C, 1, 2, 1e-6, 1e-6, 1.0, 1, 1, 1, 1, C, C, C)
        n = lib.basa_gated_norm_bwd_workspace_size(ctypes.byref(p))
        assert n % 256 == 0 and n >= 9 * 4 * C  # of one CTA: two modulations' three sums, three of the weights
        return n
    for norm in (1, 2):
        for H, Hkv, d in ((1, 1, 32), (12, 4, 128), (40, 40, 128), (128, 2, 128), (8, 8, 64)):
            sizes = [rope(norm, H, Hkv, d, t) for t in (1, 7, 100, 1000, 30000)]
            assert sizes[0] <= sizes[1] < sizes[-1], (norm, H, Hkv, d, sizes)
    for C in (8, 264, 5120, 8192):
        sizes = [border(r, 1, C) for r in (1, 4, 100, 3000, 100000)]
        assert sizes[0] <= sizes[1] < sizes[-1], (C, sizes)
    assert border(100, 1, 512) > border(100, 1, 256)
