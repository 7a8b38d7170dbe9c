"""GPU parity of the calls around the attention (qkv_rope, gated_norm and their
backwards) against their formulas in 64 bits, element by element.

Tolerances.  A result computed in fp32 from exact inputs is off by at most
K * 2^-24 times the sum of the magnitudes it was formed from, K counting the
roundings on the longest chain: a row's sum adds at most 32 values in a thread,
5 times over a warp's lanes and 20 times over a CTA's warps, and about ten
further roundings stand around it, so K = 64 + 2.  A column sum of a gradient adds
along a thread's rows (at most 28 in these cases), the CTA's 8 warps, and
partial rows of every CTA (at most 1776 in 32 chains or more, each of at most 56,
joined by 32 or fewer): K = 128.  Each rounding to the output's type adds half a step of the value, and
for e4m3 no less than half its smallest step, 2^-10."""
import math

import pytest
import torch

import oracle
from gpu_util import assert_close, oracle_params

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K_ROW, K_COL = 66, 128
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def basa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_diffusion_basa_b200 import build
    build.build()
    import sparse_attention_diffusion_basa_b200 as m
    oracle.build_oracle()
    return m


def rnd(seed, *shape, dtype=F32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def half_step(ref, dtype):
    """Half a rounding step of dtype at the value ref."""
    t = ref.abs() * (torch.finfo(dtype).eps / 2)
    return t.clamp_min(2.0 ** -10) if dtype == E4 else t


def check(got, ref, mag, k, what):
    """|got - ref| <= k 2^-24 mag + the rounding of ref (and of that error) to got's type."""
    g = got.double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), what
    tol = k * U * mag
    tol = tol + half_step(ref.abs() + tol, got.dtype)
    worst = ((g - ref).abs() / tol.clamp_min(1e-300)).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.3g} of the bound"


# ---------------------------------------------------------------------------
# qkv_rope in 64 bits
# ---------------------------------------------------------------------------
def turn64(x, cs, axes, layout):
    """x turned by cs [T, Hg, Wg, pairs, 2] and the magnitudes it was formed from."""
    p = sum(axes) // 2
    c, s = cs[..., 0].unsqueeze(3), cs[..., 1].unsqueeze(3)
    out, mag = x.clone(), x.abs()
    if layout == "pairs":
        ia, ib = slice(0, 2 * p, 2), slice(1, 2 * p, 2)
    else:
        ia, ib = slice(0, p), slice(p, 2 * p)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    both = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    mag[..., ia], mag[..., ib] = both
    return out, mag


def table64(table, grid, axes):
    """The table's pairs beside every token [T, Hg, Wg, pairs, 2]."""
    (T, Hg, Wg), n = grid, [a // 2 for a in axes]
    t, h, w = table.double().split([T * n[0], Hg * n[1], Wg * n[2]])
    return torch.cat([t.view(T, 1, 1, n[0], 2).expand(T, Hg, Wg, n[0], 2),
                      h.view(1, Hg, 1, n[1], 2).expand(T, Hg, Wg, n[1], 2),
                      w.view(1, 1, Wg, n[2], 2).expand(T, Hg, Wg, n[2], 2)], 3)


def norm_dims(norm):
    return (-1,) if norm == "head" else (-2, -1)


def w64(w, x, norm):
    if w is None:
        return torch.ones((), dtype=torch.float64, device=x.device)
    return w.double() if norm == "head" else w.double().view(x.shape[-2], x.shape[-1])


def rope64(x, w, cs, axes, layout, norm, eps):
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(norm_dims(norm), keepdim=True) + eps) * w64(w, x, norm)
    return turn64(x, cs, axes, layout)


def rope_bwd64(g, x, w, cs, axes, layout, norm, eps):
    """(dx, its magnitudes, dw, its magnitudes)."""
    back = torch.stack([cs[..., 0], -cs[..., 1]], -1)
    gn, mag = turn64(g.double(), back, axes, layout)
    if not norm:
        return gn, mag, None, None
    x, dims, wd = x.double(), norm_dims(norm), w64(w, x, norm)
    r = 1 / torch.sqrt((x * x).mean(dims, keepdim=True) + eps)
    dx = r * (wd * gn - x * r * r * (wd * gn * x).mean(dims, keepdim=True))
    dmag = r * ((wd * mag).abs() + x.abs() * r * r * (wd * mag * x).abs().mean(dims, keepdim=True))
    over = tuple(range(5 if norm == "head" else 4))
    return dx, dmag, (gn * x * r).sum(over).reshape(-1), (mag * x * r).abs().sum(over).reshape(-1)


ROPE = [
    # B, grid, H, Hkv, d, axes, norm, layout, dtype, out, weights, fused, seed
    (1, (1, 16, 16), 2, 2, 64, (0, 32, 32), "head", "halves", F32, F32, F32, False, 1),
    (1, (1, 8, 9), 24, 24, 128, (16, 56, 56), "head", "pairs", BF, BF, BF, True, 2),
    (2, (3, 5, 7), 5, 5, 128, (44, 42, 42), "token", "pairs", BF, BF, F32, True, 3),
    (2, (3, 5, 7), 6, 2, 128, (44, 42, 42), "token", "halves", F32, F32, BF, False, 4),
    (1, (1, 1, 1), 1, 1, 32, (0, 0, 32), "head", "pairs", BF, BF, None, False, 5),
    (1, (1, 1, 1), 12, 4, 32, (0, 0, 16), "token", "halves", BF, BF, F32, True, 6),
    (3, (2, 3, 11), 3, 1, 32, (2, 6, 10), "head", "pairs", BF, BF, F32, True, 7),
    (1, (4, 6, 5), 9, 3, 64, (2, 10, 20), "head", "halves", BF, BF, BF, True, 8),
    (1, (2, 6, 5), 40, 40, 128, (44, 42, 42), "token", "pairs", BF, BF, BF, False, 9),
    (1, (1, 6, 5), 128, 8, 128, (0, 64, 64), "token", "halves", BF, BF, BF, False, 10),
    (1, (1, 6, 5), 128, 128, 128, (0, 64, 64), "token", "pairs", F32, F32, F32, False, 19),
    (1, (1, 4, 7), 4, 4, 128, (0, 0, 0), "head", "pairs", BF, BF, F32, True, 11),
    (1, (1, 4, 7), 4, 2, 64, (0, 20, 44), None, "pairs", BF, BF, None, True, 12),
    (2, (2, 3, 5), 7, 7, 128, (32, 48, 48), None, "halves", F32, F32, None, False, 13),
    (1, (1, 9, 10), 3, 3, 64, (0, 32, 32), None, "halves", BF, BF, None, True, 14),
    (1, (1, 45, 31), 33, 11, 64, (0, 24, 40), "head", "pairs", BF, BF, BF, True, 15),
    # a token's heads shared between CTAs
    (1, (1, 6, 7), 40, 10, 128, (16, 56, 56), "head", "pairs", BF, BF, BF, True, 20),
    (1, (2, 3, 2), 200, 100, 32, (4, 12, 16), "head", "halves", BF, BF, F32, False, 21),
    (1, (1, 2, 5), 72, 72, 64, (0, 32, 32), None, "pairs", F32, F32, None, False, 22),
    # e4m3 outputs
    (1, (1, 8, 9), 8, 2, 128, (16, 56, 56), "head", "pairs", BF, E4, BF, True, 16),
    (2, (2, 3, 5), 4, 4, 128, (32, 48, 48), "token", "halves", BF, E4, F32, False, 17),
    (1, (1, 8, 3), 2, 2, 32, (0, 16, 16), None, "pairs", F32, E4, None, True, 18),
]


def rope_inputs(case):
    B, grid, H, Hkv, d, axes, norm, layout, dtype, out, wt, fused, seed = case
    lead = (B, *grid)
    if fused:
        whole = rnd(seed, *lead, (H + 2 * Hkv) * d, dtype=dtype, std=1.5)
        q, k, v = (t.view(*lead, -1, d) for t in whole.split([H * d, Hkv * d, Hkv * d], -1))
    else:
        q, k, v = (rnd(seed + 100 * i, *lead, n, d, dtype=dtype, std=1.5) for i, n in enumerate((H, Hkv, Hkv)))
    qw = kw = None
    if wt is not None:
        n = (d, d) if norm == "head" else (H * d, Hkv * d)
        qw, kw = (rnd(seed + 200 + i, m, dtype=wt, std=0.3, mean=1.0) for i, m in enumerate(n))
    return q, k, v, qw, kw


@pytest.mark.parametrize("case", ROPE, ids=lambda c: str(c[-1]))
def test_rope_forward(basa, case):
    B, grid, H, Hkv, d, axes, norm, layout, dtype, out, wt, fused, seed = case
    q, k, v, qw, kw = rope_inputs(case)
    table = basa.rope_table(grid, axes, 1e4, (3.0, -2.5, 0.0), (1.0, 0.5, 1.0))
    cs = table64(table, grid, axes)
    eps = 1e-5
    descale = (0.05, 0.04, 0.03) if out == E4 else (0.0, 0.0, 0.0)
    got = basa.qkv_rope(q, k, v, table, axes, layout=layout, norm=norm, q_weight=qw, k_weight=kw, eps=eps,
                        out_dtype=out, descale=descale)
    torch.cuda.synchronize()
    for i, (o, x, w) in enumerate(zip(got, (q, k, v), (qw, kw, None))):
        assert o.dtype == out and o.is_contiguous()
        if i < 2:
            ref, mag = rope64(x, w, cs, axes, layout, norm, eps)
        else:
            ref, mag = x.double(), x.double().abs()
        if out == E4:
            ref, mag = ref / descale[i], mag / descale[i]
            assert ref.abs().max() < 448
        elif i == 2:
            assert torch.equal(o, x)
        check(o, ref, mag, K_ROW, "qkv"[i])
    # without v, and the same bits again
    again = basa.qkv_rope(q, k, None, table, axes, layout=layout, norm=norm, q_weight=qw, k_weight=kw, eps=eps,
                          out_dtype=out, descale=descale)
    assert again[2] is None
    for a, b in zip(again[:2], got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("case", [c for c in ROPE if c[9] != E4], ids=lambda c: str(c[-1]))
def test_rope_backward(basa, case):
    B, grid, H, Hkv, d, axes, norm, layout, dtype, out, wt, fused, seed = case
    q, k, v, qw, kw = rope_inputs(case)
    table = basa.rope_table(grid, axes, 1e4, (3.0, -2.5, 0.0), (1.0, 0.5, 1.0))
    cs = table64(table, grid, axes)
    eps, lead = 1e-5, (B, *grid)
    gq, gk, gv = (rnd(seed + 300 + i, *lead, n, d, dtype=dtype) for i, n in enumerate((H, Hkv, Hkv)))
    into = None
    if fused:
        whole = torch.empty(*lead, (H + 2 * Hkv) * d + 8, dtype=dtype, device="cuda").fill_(7.0)
        into = [t.view(*lead, -1, d) for t in whole[..., 8:].split([H * d, Hkv * d, Hkv * d], -1)]
    args = dict(layout=layout, norm=norm, q_weight=qw, k_weight=kw, eps=eps)
    dq, dk, dv, dqw, dkw = basa.qkv_rope_bwd(gq, gk, gv, q, k, table, axes, out=into, **args)
    torch.cuda.synchronize()
    assert torch.equal(dv, gv)
    if fused:
        assert dq.data_ptr() == into[0].data_ptr()
        assert (whole[..., :8] == 7.0).all()
    for g, x, w, dx, dw, name in ((gq, q, qw, dq, dqw, "q"), (gk, k, kw, dk, dkw, "k")):
        ref, mag, wref, wmag = rope_bwd64(g, x, w, cs, axes, layout, norm, eps)
        check(dx, ref, mag, K_ROW, f"d{name}")
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == w.dtype and dw.shape == w.shape
            check(dw, wref, wmag, K_COL, f"d{name}_weight")
    again = basa.qkv_rope_bwd(gq, gk, None, q if norm else None, k if norm else None, table, axes, **args)
    for a, b in zip((again[0], again[1], again[3], again[4]), (dq, dk, dqw, dkw)):
        assert (a is None and b is None) or torch.equal(a, b)
    assert again[2] is None


@pytest.mark.parametrize("norm,H,Hkv", [("head", 24, 8), ("token", 12, 3), ("token", 40, 40), (None, 5, 5)])
def test_rope_many_tokens(basa, norm, H, Hkv):
    """More tokens than warps and teams at a time: each takes several, across rows and frames."""
    B, grid, d, axes = 2, (5, 31, 67), 128, (44, 42, 42)
    q, k = rnd(1, B, *grid, H, d, dtype=BF), rnd(2, B, *grid, Hkv, d, dtype=BF)
    gq, gk = rnd(3, B, *grid, H, d, dtype=BF), rnd(4, B, *grid, Hkv, d, dtype=BF)
    n = {"head": (d, d), "token": (H * d, Hkv * d)}.get(norm)
    qw, kw = (rnd(5 + i, m, mean=1.0, std=0.3) for i, m in enumerate(n)) if norm else (None, None)
    table = basa.rope_table(grid, axes)
    cs = table64(table, grid, axes)
    args = dict(norm=norm, q_weight=qw, k_weight=kw)
    qo, ko, _ = basa.qkv_rope(q, k, None, table, axes, **args)
    dq, dk, _, dqw, dkw = basa.qkv_rope_bwd(gq, gk, None, q, k, table, axes, **args)
    for x, g, w, o, dx, dw, name in ((q, gq, qw, qo, dq, dqw, "q"), (k, gk, kw, ko, dk, dkw, "k")):
        ref, mag = rope64(x, w, cs, axes, "pairs", norm, 1e-6)
        check(o, ref, mag, K_ROW, name)
        ref, mag, wref, wmag = rope_bwd64(g, x, w, cs, axes, "pairs", norm, 1e-6)
        check(dx, ref, mag, K_ROW, f"d{name}")
        if w is not None:
            # a thread adds at most 20770 tokens' heads / (148 CTAs * 4 warps * 4 heads a step) < 180 terms,
            # and at most 2368 partial rows in 128 chains of 19, joined by 12
            check(dw, wref, wmag, 180 + 8 + 19 + 12 + K_ROW, f"d{name}_weight")


def test_rope_gradients_against_differences(basa):
    """d/de of sum(gradient * forward(inputs + e direction)), the forward in 64 bits."""
    B, grid, H, Hkv, d, axes = 1, (2, 3, 4), 4, 2, 64, (16, 24, 24)
    table = basa.rope_table(grid, axes)
    cs = table64(table, grid, axes)
    for norm, layout in (("head", "halves"), ("token", "pairs"), (None, "pairs")):
        q, k = rnd(1, B, *grid, H, d), rnd(2, B, *grid, Hkv, d)
        gq, gk = rnd(3, B, *grid, H, d), rnd(4, B, *grid, Hkv, d)
        n = {"head": (d, d), "token": (H * d, Hkv * d), None: (0, 0)}[norm]
        qw, kw = (rnd(5 + i, m, mean=1.0, std=0.3) for i, m in enumerate(n)) if norm else (None, None)
        dq, dk, _, dqw, dkw = basa.qkv_rope_bwd(gq, gk, None, q, k, table, axes, layout=layout, norm=norm,
                                                q_weight=qw, k_weight=kw)
        for x, w, g, dx, dw in ((q, qw, gq, dq, dqw), (k, kw, gk, dk, dkw)):
            f = lambda x_, w_: (g.double() * rope64(x_, w_, cs, axes, layout, norm, 1e-6)[0]).sum()  # noqa: E731
            e, x64, w64_ = 1e-6, x.double(), None if w is None else w.double()
            v = rnd(9, *x.shape).double()
            num = (f(x64 + e * v, w64_) - f(x64 - e * v, w64_)) / (2 * e)
            # differences: error e^2 and 2^-53 / e, both below 1e-9 of the terms' sum; the kernel's K_ROW 2^-24
            scale = (dx.double() * v).abs().sum() + (g.double().abs() * x64.abs()).sum()
            assert abs(num - (dx.double() * v).sum()) <= K_ROW * U * scale
            if w is not None:
                v = rnd(10, *w.shape).double()
                num = (f(x64, w64_ + e * v) - f(x64, w64_ - e * v)) / (2 * e)
                assert abs(num - (dw.double() * v).sum()) <= K_COL * U * ((dw.double() * v).abs().sum() + scale)


def test_rope_table_values(basa):
    """Far and fractional positions against 64 bits: the fp32 rounding alone, 2^-24 relative,
    beside the 64-bit angle's own error of 2^-52 of the angle."""
    grid, axes, theta = (3, 70, 9), (16, 56, 40), 5000.0
    start, step = (1e5, -34.5, 0.25), (7.0, 1.0, 0.125)
    got = basa.rope_table(grid, axes, theta, start, step).double()
    off = 0
    for G, a, s, e in zip(grid, axes, start, step):
        f = theta ** (-torch.arange(0, a, 2, dtype=torch.float64, device="cuda") / a)
        ang = (s + e * torch.arange(G, dtype=torch.float64, device="cuda"))[:, None] * f
        ref = torch.stack([ang.cos(), ang.sin()], -1).reshape(-1, 2)
        part = got[off:off + ref.shape[0]]
        assert ((part - ref).abs() <= U * ref.abs() + 8 * 2.0 ** -52 * ang.abs().reshape(-1, 1) + 1e-30).all()
        off += ref.shape[0]
    assert off == got.shape[0]
    out = torch.empty_like(got, dtype=F32)
    assert basa.rope_table(grid, axes, theta, start, step, out=out) is out
    assert torch.equal(out.double(), got)
    assert basa.rope_table((1, 4, 4), (0, 0, 0)).shape == (0, 2)
    with pytest.raises(ValueError, match="table"):
        basa.rope_table(grid, axes, out=out[:-1])


def test_rope_text_positions_of_zero_change_nothing(basa):
    """Text tokens at position 0 on every axis: rotation by zero, exactly."""
    q, k = rnd(1, 2, 7, 3, 128, dtype=BF), rnd(2, 2, 7, 3, 128, dtype=BF)
    table = basa.rope_table((1, 1, 7), (0, 0, 128), step=(0.0, 0.0, 0.0))
    qo, ko, _ = basa.qkv_rope(q, k, None, table, (0, 0, 128))
    assert torch.equal(qo, q) and torch.equal(ko, k)


@pytest.mark.parametrize("norm", [None, "head", "token"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_in_place(basa, norm, layout):
    grid, axes = (2, 4, 5), (32, 48, 48)
    table = basa.rope_table(grid, axes)
    q, k, v = (rnd(i, 2, *grid, n, 128, dtype=BF) for i, n in enumerate((6, 3, 3)))
    args = dict(layout=layout, norm=norm)
    want = basa.qkv_rope(q, k, v, table, axes, **args)
    qc, kc, vc = q.clone(), k.clone(), v.clone()
    got = basa.qkv_rope(qc, kc, vc, table, axes, out=(qc, kc, vc), **args)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    gq, gk = rnd(8, *q.shape, dtype=BF), rnd(9, *k.shape, dtype=BF)
    want = basa.qkv_rope_bwd(gq, gk, None, q, k, table, axes, **args)
    got = basa.qkv_rope_bwd(gq, gk, None, q, k, table, axes, out=(gq, gk, None), **args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rope_special_values(basa):
    """NaN and infinity stay in their own head (or token); e4m3 outputs stop at 448."""
    grid, axes = (1, 4, 4), (0, 32, 32)
    table = basa.rope_table(grid, axes)
    q, k = rnd(1, 1, *grid, 4, 64, dtype=BF), rnd(2, 1, *grid, 4, 64, dtype=BF)
    for norm in ("head", "token"):
        clean, _, _ = basa.qkv_rope(q, k, None, table, axes, norm=norm)
        bad = q.clone()
        bad[0, 0, 1, 2, 3, 5] = float("nan")
        bad[0, 0, 3, 0, 1, 7] = float("inf")
        got, _, _ = basa.qkv_rope(bad, k, None, table, axes, norm=norm)
        same = torch.ones(1, *grid, 4, dtype=torch.bool, device="cuda")
        if norm == "head":
            same[0, 0, 1, 2, 3] = same[0, 0, 3, 0, 1] = False
        else:
            same[0, 0, 1, 2] = same[0, 0, 3, 0] = False
        assert torch.equal(got[same], clean[same])
        assert torch.isnan(got[0, 0, 1, 2, 3]).all()
        zero, _, _ = basa.qkv_rope(torch.zeros_like(q), k, None, table, axes, norm=norm)
        assert (zero == 0).all()
    v = torch.zeros_like(k)
    v[0, 0, 0, 0, 0, :4] = torch.tensor([1000.0, -1000.0, float("nan"), 3.0])
    _, _, vo = basa.qkv_rope(q, k, v, table, axes, out_dtype=E4)
    assert vo[0, 0, 0, 0, 0, :2].float().tolist() == [448.0, -448.0]
    assert torch.isnan(vo[0, 0, 0, 0, 0, 2].float()) and vo[0, 0, 0, 0, 0, 3].float() == 3.0


def test_rope_empty(basa):
    w = torch.ones(64, device="cuda")
    for shape in ((0, 1, 4, 4, 2, 64), (1, 1, 0, 4, 2, 64)):
        q = torch.empty(shape, device="cuda")
        table = basa.rope_table((1, shape[2], 4), (0, 32, 32))
        out = basa.qkv_rope(q, q, q, table, (0, 32, 32), norm="head", q_weight=w, k_weight=w)
        assert all(o.shape == q.shape for o in out)
        g = basa.qkv_rope_bwd(q, q, q, q, q, table, (0, 32, 32), norm="head", q_weight=w, k_weight=w)
        assert (g[3] == 0).all() and (g[4] == 0).all()


def test_rope_rows_beyond_32_bits(basa):
    """Slices of a buffer whose last rows lie past 2^31 elements; what lies between stays."""
    n, ld, H, d = 70000, 32768, 2, 64
    buf = torch.empty(n, ld, dtype=BF, device="cuda")
    q = buf[:, 1024:1024 + H * d].unflatten(1, (H, d))[None]
    k = buf[:, 8192:8192 + H * d].unflatten(1, (H, d))[None]
    q.copy_(rnd(1, *q.shape, dtype=BF))
    k.copy_(rnd(2, *k.shape, dtype=BF))
    axes, grid = (0, 0, 64), (1, 1, n)
    table = basa.rope_table(grid, axes)
    for norm in ("head", "token"):
        got = basa.qkv_rope(q, k, None, table, axes, norm=norm)
        want = basa.qkv_rope(q.contiguous(), k.contiguous(), None, table, axes, norm=norm)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        want = basa.qkv_rope_bwd(*want, q.contiguous(), k.contiguous(), table, axes, norm=norm)
        guard = buf[-1, 1024 + H * d:8192].clone()
        dst = basa.qkv_rope_bwd(*got, q.contiguous(), k.contiguous(), table, axes, norm=norm, out=(q, k, None))
        assert torch.equal(dst[0], want[0]) and torch.equal(dst[1], want[1])
        assert torch.equal(buf[-1, 1024 + H * d:8192].view(torch.int16), guard.view(torch.int16))


# ---------------------------------------------------------------------------
# gated_norm in 64 bits
# ---------------------------------------------------------------------------
def stats64(x, kind, eps):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    return mean, 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)


def beside(m, rows, like):
    """A modulation's row beside each of `rows` tokens [rows, C]; None: the neutral value."""
    if m is None:
        return like
    m = m.double().reshape(-1, m.shape[-1])
    return m.repeat_interleave(rows // m.shape[0], 0)


def border64(x, y, p, norm, post, eps, post_eps, res):
    """x_out, h, stats and the magnitudes behind x_out and h; rows [n, C]."""
    n, C = x.shape
    one, zero = torch.ones((), dtype=torch.float64, device=x.device), torch.zeros((), dtype=torch.float64, device=x.device)
    w64_ = lambda t, d: d if t is None else t.double()  # noqa: E731
    none = torch.zeros(n, 1, dtype=torch.float64, device=x.device)
    pm, ps = none, none
    mag = x.abs()
    if y is not None:
        u, umag = y, y.abs()
        if post:
            pm, ps = stats64(y, post, post_eps)
            u = (y - pm) * ps
            umag = (1 + u.abs()) * (1 + y.abs().amax(-1, keepdim=True) * ps)
        G = w64_(p["post_weight"], one) * beside(p["gate"], n, one)
        mag = (res * x).abs() + G.abs() * umag
        x = res * x + G * u
    if not norm:
        return x, None, torch.cat([none, none, pm, ps], -1), mag, None
    m, s = stats64(x, norm, eps)
    xh = (x - m) * s
    w, b = w64_(p["weight"], one), w64_(p["bias"], zero)
    scale, shift = beside(p["scale"], n, zero), beside(p["shift"], n, zero)
    h = (xh * w + b) * (1 + scale) + shift
    far = 1 + mag.amax(-1, keepdim=True) * s
    hmag = w.abs() * (1 + scale.abs()) * (1 + xh.abs()) * far + b.abs() * (1 + scale.abs()) + shift.abs()
    return x, h, torch.cat([m, s, pm, ps], -1), mag, hmag


BORDER = [
    # lead, C, (x, y) types, modulation dims, mod type, weight type, which, norm, post, res, seed
    ((2, 5, 7), 64, (BF, BF), 1, BF, None, "gate scale shift", "layer", None, 1.0, 1),
    ((3, 4, 3, 5), 1000, (F32, F32), 1, F32, F32, "gate scale shift weight bias post_weight", "layer", "rms", 1.0, 2),
    ((3, 4, 3, 5), 1000, (F32, BF), 2, F32, BF, "gate scale shift weight post_weight", "rms", "layer", 0.5, 3),
    ((1, 1), 8, (BF, BF), 0, BF, BF, "gate weight bias", "layer", "rms", 1.0, 4),
    ((2, 9), 8192, (F32, F32), 1, BF, F32, "gate scale shift weight bias", "layer", "layer", -1.5, 5),
    ((2, 40), 5120, (F32, BF), 1, BF, None, "gate scale shift", "layer", None, 1.0, 6),
    ((2, 40), 5120, (BF, BF), 2, BF, F32, "gate scale shift weight bias post_weight", "rms", "rms", 1.0, 7),
    ((5, 6), 4104, (BF, BF), 1, F32, BF, "scale shift weight bias", "layer", None, 1.0, 8),
    ((2, 3, 6), 5128, (BF, BF), 3, BF, BF, "gate shift post_weight", "rms", "layer", 2.0, 9),
    ((4, 31), 264, (F32, BF), 0, F32, F32, "scale bias", "layer", "rms", 1.0, 10),
    ((700, 5), 72, (BF, BF), 1, BF, F32, "gate scale shift weight bias post_weight", "layer", "rms", 1.0, 11),
    ((3, 331), 1152, (BF, BF), 1, BF, None, "", "rms", None, 1.0, 12),
    ((2, 17), 1536, (BF, BF), 1, BF, BF, "gate post_weight", None, "rms", 1.0, 13),
    ((2, 17), 1536, (F32, BF), 1, F32, BF, "gate", None, None, 0.25, 14),
    ((2, 17), 1536, (F32, F32), 0, F32, BF, "", None, None, 1.0, 15),
    ((2, 19), 2048, (BF, None), 1, BF, BF, "scale shift weight bias", "layer", None, 1.0, 16),
    ((2, 19), 640, (F32, None), 1, BF, F32, "scale weight", "rms", None, 1.0, 17),
    ((1, 3), 8192, (BF, BF), 1, BF, BF, "gate scale shift weight bias post_weight", "layer", "rms", 1.0, 18),
]
IDS = lambda c: str(c[-1])  # noqa: E731


def border_inputs(case):
    lead, C, (xt, yt), nmod, mt, wt, which, norm, post, res, seed = case
    x = rnd(seed, *lead, C, dtype=xt, std=2.0, mean=0.7)
    y = rnd(seed + 50, *lead, C, dtype=yt, mean=0.3) if yt is not None else None
    slices = rnd(seed + 100, *lead[:nmod], 3, C, dtype=mt, std=0.5)  # one modulation output
    p = dict.fromkeys(("gate", "scale", "shift", "weight", "bias", "post_weight"))
    for i, k in enumerate(("gate", "scale", "shift")):
        if k in which.split():
            p[k] = slices[..., i, :]
    for i, k in enumerate(("weight", "bias", "post_weight")):
        if k in which.split():
            p[k] = rnd(seed + 200 + i, C, dtype=wt, std=0.3, mean=1.0 if k != "bias" else 0.0)
    return x, y, p


@pytest.mark.parametrize("case", BORDER, ids=IDS)
def test_border_forward(basa, case):
    lead, C, (xt, yt), nmod, mt, wt, which, norm, post, res, seed = case
    x, y, p = border_inputs(case)
    n = x.numel() // C
    f = lambda: basa.gated_norm(x, y, norm=norm, post_norm=post, eps=1e-5, post_eps=1e-6, res_scale=res,  # noqa: E731
                                return_stats=True, **p)
    xo, h, st = f()
    torch.cuda.synchronize()
    rx, rh, rs, mag, hmag = border64(x.double().view(n, C), None if y is None else y.double().view(n, C), p, norm,
                                     post, 1e-5, 1e-6, res)
    if y is None:
        assert xo is x
    else:
        assert xo.dtype == xt
        check(xo.view(n, C), rx, mag, K_ROW, "x_out")
    if norm is None:
        assert h is None
    else:
        assert h.dtype == (yt or xt)
        check(h.view(n, C), rh, hmag, K_ROW, "h")
    # a mean is off by K of the mean magnitude, a deviation's inverse by K (1 + magnitude * inverse) of itself
    for i, a in ((0, mag), (2, None if y is None else y.double().view(n, C).abs())):
        if a is None:
            continue
        top = a.amax(-1)
        tol = K_ROW * U * torch.stack([top, rs[:, i + 1] * (1 + top * rs[:, i + 1])], -1)
        assert ((st.view(n, 4).double()[:, i:i + 2] - rs[:, i:i + 2]).abs() <= tol).all()
    for a, b in zip(f(), (xo, h, st)):
        assert (a is None and b is None) or torch.equal(a, b)


def border_bwd64(gh, gx, x, y, st, p, norm, post, res):
    """Every gradient with the magnitudes behind it; st as given to the kernel."""
    n, C = (gx if gx is not None else gh).shape
    dev = st.device
    one, zero = torch.ones((), dtype=torch.float64, device=dev), torch.zeros((), dtype=torch.float64, device=dev)
    wd = lambda t, d: d if t is None else t.double()  # noqa: E731
    groups = next((p[k].numel() // C for k in ("gate", "scale", "shift") if p[k] is not None), 1)
    per = lambda v: v.view(groups, n // groups, C).sum(1)  # noqa: E731
    out = {}
    t = gx if gx is not None else torch.zeros(n, C, dtype=torch.float64, device=dev)
    tm = t.abs()
    if norm:
        m, s = st[:, 0:1], st[:, 1:2]
        xh = (x - m) * s
        xm = (x.abs() + m.abs()) * s              # what xh was formed from
        w, b = wd(p["weight"], one), wd(p["bias"], zero)
        scale = beside(p["scale"], n, zero)
        a = gh * (1 + scale) * w
        am = gh.abs() * (1 + scale.abs()) * w.abs()
        c1 = a.mean(-1, keepdim=True) if norm == "layer" else 0.0
        t = t + s * (a - c1 - xh * (a * xh).mean(-1, keepdim=True))
        tm = tm + s * (am + am.mean(-1, keepdim=True) + xm * (am * xm).mean(-1, keepdim=True))
        g1 = gh * (1 + scale)
        g1m = gh.abs() * (1 + scale.abs())
        out["dscale"] = per(gh * (xh * w + b)), per(gh.abs() * (xm * w.abs() + b.abs()))
        out["dshift"] = per(gh), per(gh.abs())
        out["dweight"] = (g1 * xh).sum(0), (g1m * xm).sum(0)
        out["dbias"] = g1.sum(0), g1m.sum(0)
    out["dx"] = res * t, abs(res) * tm
    if y is not None:
        gate, pw = beside(p["gate"], n, one), wd(p["post_weight"], one)
        e, em = t * gate * pw, tm * (gate * pw).abs()
        yh, ym = y, y.abs()
        if post:
            pm, ps = st[:, 2:3], st[:, 3:4]
            yh = (y - pm) * ps
            ym = (y.abs() + pm.abs()) * ps
        out["dgate"] = per(t * yh * pw), per(tm * ym * pw.abs())
        out["dpost_weight"] = (t * yh * gate).sum(0), (tm * ym * gate.abs()).sum(0)
        if post:
            c1 = e.mean(-1, keepdim=True) if post == "layer" else 0.0
            dy = ps * (e - c1 - yh * (e * yh).mean(-1, keepdim=True))
            dym = ps * (em + em.mean(-1, keepdim=True) + ym * (em * ym).mean(-1, keepdim=True))
        else:
            dy, dym = e, em
        out["dy"] = dy, dym
    return out


def border_grads(basa, case, with_gx=True):
    lead, C, (xt, yt), nmod, mt, wt, which, norm, post, res, seed = case
    x, y, p = border_inputs(case)
    n = x.numel() // C
    st = [torch.zeros(n, 1, dtype=torch.float64, device="cuda")] * 4
    if norm:
        st[0:2] = stats64(x.double().view(n, C), norm, 1e-5)
    if post:
        st[2:4] = stats64(y.double().view(n, C), post, 1e-6)
    st = torch.cat(st, -1).float().view(*lead, 4).contiguous()
    gh = rnd(seed + 300, *lead, C, dtype=yt or xt, mean=0.2) if norm else None
    gx = rnd(seed + 301, *lead, C, dtype=xt) if with_gx or not norm else None
    got = basa.gated_norm_bwd(gh, x if norm else None, st if norm or post else None, y, gx, norm=norm, post_norm=post,
                              res_scale=res, **p)
    torch.cuda.synchronize()
    v = lambda t: None if t is None else t.double().view(n, C)  # noqa: E731
    return got, border_bwd64(v(gh), v(gx), v(x), v(y), st.double().view(n, 4), p, norm, post, res), p


@pytest.mark.parametrize("case", BORDER, ids=IDS)
@pytest.mark.parametrize("with_gx", [True, False])
def test_border_backward(basa, case, with_gx):
    C = case[1]
    got, ref, p = border_grads(basa, case, with_gx)
    for name in got._fields:
        g = getattr(got, name)
        param = p.get(name[1:])
        if name not in ("dx", "dy") and param is None:
            assert g is None, name
            continue
        if name == "dy" and case[2][1] is None:
            assert g is None
            continue
        if name not in ("dx", "dy"):
            assert g.dtype == param.dtype and g.shape == param.shape, name
        want, mag = ref[name]
        check(g.reshape(want.shape), want, mag, K_ROW if name in ("dx", "dy") else K_COL + K_ROW, name)


@pytest.mark.parametrize("case", [c for c in BORDER if c[-1] in (2, 3, 7, 11, 12)], ids=IDS)
def test_border_backward_gives_the_same_bits(basa, case):
    a, _, _ = border_grads(basa, case)
    b, _, _ = border_grads(basa, case)
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x, y)


# groups of tokens that begin and end inside, at and across a CTA's run of rows
@pytest.mark.parametrize("lead,nmod", [((1, 1, 1), 2), ((1, 4000), 1), ((2, 2000), 1), ((5, 800), 1), ((400, 10), 1),
                                       ((1333, 3), 1), ((1, 3999), 2), ((7, 9, 61), 2), ((3, 1301), 0)])
@pytest.mark.parametrize("C", [256, 5120])
def test_border_groups(basa, lead, nmod, C):
    case = (lead, C, (BF, BF), nmod, F32, F32, "gate scale shift weight bias post_weight", "layer", "rms", 1.0, 77)
    x, y, p = border_inputs(case)
    n = x.numel() // C
    xo, h = basa.gated_norm(x, y, norm="layer", post_norm="rms", eps=1e-5, **p)
    rx, rh, _, mag, hmag = border64(x.double().view(n, C), y.double().view(n, C), p, "layer", "rms", 1e-5, 1e-6, 1.0)
    check(xo.view(n, C), rx, mag, K_ROW, "x_out")
    check(h.view(n, C), rh, hmag, K_ROW, "h")
    got, ref, p = border_grads(basa, case)
    for name in ("dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight"):
        want, mag = ref[name]
        check(getattr(got, name).reshape(want.shape), want, mag, K_COL + K_ROW, name)


def test_border_gradients_against_differences(basa):
    lead, C = (2, 3, 5), 96
    for norm, post, res in (("layer", "rms", 1.0), ("rms", "layer", 0.5), ("layer", None, 1.0), (None, "rms", 2.0)):
        which = "gate post_weight" if post else "gate"
        which += " scale shift weight bias" if norm else ""
        case = (lead, C, (F32, F32), 1, F32, F32, which, norm, post, res, 31)
        x, y, p = border_inputs(case)
        xo, h, st = basa.gated_norm(x, y, norm=norm, post_norm=post, eps=1e-5, res_scale=res, return_stats=True, **p)
        gh, gx = rnd(5, *lead, C), rnd(6, *lead, C)
        g = basa.gated_norm_bwd(gh if norm else None, xo, st, y, gx, norm=norm, post_norm=post, res_scale=res, **p)
        n = 30
        leaves = {"x": x, "y": y, **{k: v for k, v in p.items() if v is not None}}

        def loss(values):
            q = {k: values.get(k) for k in p}
            rx, rh, _, _, _ = border64(values["x"].view(n, C), values["y"].view(n, C), q, norm, post, 1e-5, 1e-6, res)
            s = (rx * gx.double().view(n, C)).sum()
            return s + (rh * gh.double().view(n, C)).sum() if norm else s
        base = {k: v.double() for k, v in leaves.items()}
        for name in leaves:
            v = rnd(7, *leaves[name].shape).double()
            e = 1e-6
            num = (loss({**base, name: base[name] + e * v}) - loss({**base, name: base[name] - e * v})) / (2 * e)
            grad = getattr(g, "d" + name).double()
            # the differences' own error is below 1e-8 of the loss terms; the kernel's K 2^-24 of the terms' sum,
            # taken as the sum of |gradient * direction| and of the loss's own terms
            scale = (grad * v).abs().sum() + gx.double().abs().sum() * 4 + gh.double().abs().sum() * 4
            assert abs(num - (grad * v).sum()) <= (K_COL + K_ROW) * U * scale, (name, norm, post)


def test_border_in_place_and_expanded(basa):
    x, y = rnd(1, 2, 33, 1024, dtype=BF), rnd(2, 2, 33, 1024, dtype=BF)
    gate = rnd(3, 1024, dtype=BF)
    want = basa.gated_norm(x, y, gate=gate)
    xc, yc = x.clone(), y.clone()
    got = basa.gated_norm(xc, yc, gate=gate, x_out=xc, h_out=yc)
    assert got[0] is xc and got[1] is yc
    assert torch.equal(xc, want[0]) and torch.equal(yc, want[1])
    scale = rnd(4, 2, 1024, dtype=BF)
    a = basa.gated_norm(x, y, gate=gate.expand(2, 1024), scale=scale)
    b = basa.gated_norm(x, y, gate=gate.expand(2, 1024).contiguous(), scale=scale)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError, match="leading dims"):
        basa.gated_norm(x, y, gate=gate, scale=scale)


def test_border_outputs_at_16_bytes(basa):
    """fp32 outputs aligned to 16 bytes but not to 32, rows that end inside a warp, guards around them."""
    n, C = 37, 712
    x, y = rnd(1, n, C), rnd(2, n, C)
    want = basa.gated_norm(x, y, post_norm="layer")
    buf = torch.full((2, n * C + 16), 9.0, device="cuda")
    outs = [b[4:4 + n * C].view(n, C) for b in buf]
    got = basa.gated_norm(x, y, post_norm="layer", x_out=outs[0], h_out=outs[1])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (buf[:, :4] == 9.0).all() and (buf[:, 4 + n * C:] == 9.0).all()


def test_border_backward_writes_nothing_else(basa):
    """The C entry on guarded buffers, with one workspace for two calls of different shapes."""
    from sparse_attention_diffusion_basa_b200 import _lib
    import ctypes
    lib = _lib.load()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for rows, groups, C in ((333, 3, 1000), (35, 7, 264)):
        f = lambda seed, *s: rnd(seed, *s, dtype=BF)  # noqa: E731
        x, y, gh, gx = (f(i, rows, C) for i in range(4))
        mods, w = [f(10 + i, groups, C) for i in range(3)], [f(20 + i, C) for i in range(3)]
        st = torch.cat([torch.zeros(rows, 1, device="cuda"), torch.ones(rows, 1, device="cuda")] * 2, 1).contiguous()
        sizes = [rows * C, rows * C, groups * C, C, C, C, groups * C, groups * C]
        bufs = [torch.full((s + 64,), 3.0, dtype=BF, device="cuda") for s in sizes]
        outs = [b[32:32 + s] for b, s in zip(bufs, sizes)]
        prm = _lib.BasaGnormParams(rows, groups, C, 1, 2, 1e-6, 1e-6, 1.0, 1, 1, 1, 1, C, C, C)
        assert lib.basa_gated_norm_bwd_workspace_size(ctypes.byref(prm)) <= ws.numel()
        p = lambda t: t.data_ptr()  # noqa: E731
        code = lib.basa_gated_norm_bwd(p(gh), p(x), p(st), p(y), p(gx), p(mods[0]), p(w[0]), p(w[1]), p(w[2]),
                                       p(mods[1]), *(p(o) for o in outs), p(ws), ctypes.byref(prm),
                                       torch.cuda.current_stream().cuda_stream)
        assert code == 0
        torch.cuda.synchronize()
        view = lambda t: t.view(groups, rows // groups, C)  # noqa: E731
        g = basa.gated_norm_bwd(view(gh), view(x), st.view(groups, -1, 4), view(y), view(gx), gate=mods[0],
                                post_weight=w[0], weight=w[1], bias=w[2], scale=mods[1], shift=mods[2],
                                norm="layer", post_norm="rms")
        for a, b in zip(g, outs):
            assert torch.equal(a.reshape(-1), b)
        for b, s in zip(bufs, sizes):
            assert (b[:32] == 3.0).all() and (b[32 + s:] == 3.0).all()
            assert torch.isfinite(b).all() and not (b[32:32 + s] == 3.0).all()


def test_border_far_mean(basa):
    """A mean a thousand deviations from zero: squares about the row's own mean keep the digits
    (the bound's factor 1 + magnitude / deviation is 2^10 here; sums of plain squares lose 2^20)."""
    x = (rnd(1, 4, 50, 2000) + 1000.0)
    _, h, st = basa.gated_norm(x, None, norm="layer", eps=1e-6, return_stats=True)
    rx, rh, rs, mag, hmag = border64(x.double().view(200, 2000), None, dict.fromkeys(
        ("gate", "scale", "shift", "weight", "bias", "post_weight")), "layer", None, 1e-6, 1e-6, 1.0)
    check(h.view(200, 2000), rh, hmag, K_ROW, "h")


def test_border_special_rows(basa):
    """A row of one value has no deviation; NaN and infinity stay in their row."""
    x, y = rnd(1, 1, 40, 512, dtype=BF), rnd(2, 1, 40, 512, dtype=BF)
    clean = basa.gated_norm(x, y, post_norm="rms")
    bad = x.clone()
    bad[0, 3, 7], bad[0, 20, 0] = float("nan"), float("inf")
    got = basa.gated_norm(bad, y, post_norm="rms")
    keep = [i for i in range(40) if i not in (3, 20)]
    assert torch.equal(got[0][0, keep], clean[0][0, keep]) and torch.equal(got[1][0, keep], clean[1][0, keep])
    assert torch.isnan(got[1][0, 3]).all()
    c = torch.full((1, 3, 512), 2.5, device="cuda", dtype=BF)
    _, h = basa.gated_norm(c, None, norm="layer")
    assert (h == 0).all()
    z = torch.zeros(1, 3, 512, device="cuda", dtype=BF)
    xo, h = basa.gated_norm(z, z, norm="rms", post_norm="rms")
    assert (xo == 0).all() and (h == 0).all()


def test_border_empty(basa):
    for shape, mod in (((0, 5, 64), (0, 64)), ((2, 0, 64), (2, 64)), ((2, 0, 64), (64,))):
        x = torch.empty(shape, device="cuda")
        gate, w = torch.ones(mod, device="cuda"), torch.ones(64, device="cuda")
        xo, h, st = basa.gated_norm(x, x, gate=gate, scale=gate, shift=gate, weight=w, bias=w, return_stats=True)
        assert xo.shape == h.shape == x.shape and st.shape == (*shape[:-1], 4)
        g = basa.gated_norm_bwd(x, x, st, x, x, gate=gate, scale=gate, shift=gate, weight=w, bias=w)
        for t in g[2:]:
            assert t is None or (t == 0).all()


def test_border_rows_beyond_32_bits(basa):
    """More than 2^31 elements: the last rows, and what lies behind them, as a small call has them."""
    n, C = 270000, 8192
    buf = torch.zeros(n + 1, C, dtype=BF, device="cuda")
    out = torch.full((n + 1, C), 5.0, dtype=BF, device="cuda")
    buf[n - 600:n].copy_(rnd(1, 600, C, dtype=BF))
    basa.gated_norm(buf[:n], None, norm="layer", h_out=out[:n])
    _, small = basa.gated_norm(buf[n - 600:n].clone(), None, norm="layer")
    assert torch.equal(out[n - 600:n], small)
    assert (out[n] == 5.0).all()


# ---------------------------------------------------------------------------
# How a program calls them
# ---------------------------------------------------------------------------
def train_step(basa, s):
    """One pass through border, preparation and both backwards; a list of tensors."""
    table = basa.rope_table(s["grid"], s["axes"])
    xo, h, st = basa.gated_norm(s["x"], s["y"], gate=s["gate"], scale=s["scale"], shift=s["shift"],
                                post_norm="rms", return_stats=True)
    q, k, v = basa.qkv_rope(s["q"], s["k"], s["v"], table, s["axes"], norm="head", q_weight=s["w"], k_weight=s["w"])
    g = basa.qkv_rope_bwd(q, k, v, s["q"], s["k"], table, s["axes"], norm="head", q_weight=s["w"], k_weight=s["w"])
    b = basa.gated_norm_bwd(h, xo, st, s["y"], s["x"], gate=s["gate"], scale=s["scale"], shift=s["shift"],
                            post_norm="rms")
    return [t for t in (table, xo, h, st, q, k, v, *g, *b) if t is not None]


def step_state(seed, n=300):
    grid, axes = (1, 6, n // 6), (0, 24, 40)
    s = {"grid": grid, "axes": axes, "x": rnd(seed, 1, n, 768, dtype=BF), "y": rnd(seed + 1, 1, n, 768, dtype=BF),
         "w": rnd(seed + 2, 64, dtype=BF, mean=1.0)}
    for i, k in enumerate(("gate", "scale", "shift")):
        s[k] = rnd(seed + 3 + i, 1, 768, dtype=BF)
    for i, (k, h) in enumerate((("q", 4), ("k", 2), ("v", 2))):
        s[k] = rnd(seed + 6 + i, 1, *grid, h, 64, dtype=BF)
    return s


def test_captured_and_replayed(basa):
    """Two captured steps and an eager one, interleaved: each graph has its own workspaces."""
    states = [step_state(10), step_state(40)]
    want = [train_step(basa, s) for s in states]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in states:
        with torch.cuda.stream(side):
            train_step(basa, s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            o = train_step(basa, s)
        graphs.append(g)
        outs.append(o)
    for o in outs:
        for t in o:
            t.view(torch.uint8).zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0].replay()
        graphs[1].replay()
        eager = train_step(basa, states[0])
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.synchronize()
    for got, ref in ((outs[0], want[0]), (outs[1], want[1]), (eager, want[0])):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # new inputs through the captured graph
    new = step_state(70)
    for k, v in states[0].items():
        if isinstance(v, torch.Tensor):
            v.copy_(new[k])
    want = train_step(basa, new)
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))


def test_streams(basa):
    """Two calls at once on two streams, given by argument and as the current one; memory that a
    call frees is not handed to another stream."""
    s1, s2 = step_state(10, 6000), step_state(40, 6000)
    want = [train_step(basa, s) for s in (s1, s2)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(a):
            r1 = train_step(basa, s1)
        with torch.cuda.stream(b):
            r2 = train_step(basa, s2)
        axes = s1["axes"]
        t = basa.rope_table(s1["grid"], axes, stream=a)
        q, k, v = basa.qkv_rope(s1["q"], s1["k"], s1["v"], t, axes, norm="head", q_weight=s1["w"], k_weight=s1["w"],
                                stream=a)
        g = basa.qkv_rope_bwd(q, k, v, s1["q"], s1["k"], t, axes, norm="head", q_weight=s1["w"], k_weight=s1["w"],
                              stream=a)
        mods = {n: s1[n] for n in ("gate", "scale", "shift")}
        xo, h, st = basa.gated_norm(s1["x"], s1["y"], post_norm="rms", return_stats=True, stream=a, **mods)
        d = basa.gated_norm_bwd(h, xo, st, s1["y"], s1["x"], post_norm="rms", stream=a, **mods)
        torch.cuda.synchronize()
        r3 = [x for x in (t, xo, h, st, q, k, v, *g, *d) if x is not None]
        for got, ref in ((r1, want[0]), (r2, want[1]), (r3, want[0])):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))


def test_refused_on_the_device(basa):
    q = rnd(1, 1, 1, 4, 4, 2, 64, dtype=BF)
    t = basa.rope_table((1, 4, 4), (0, 32, 32))
    ok = dict(table=t, axes=(0, 32, 32))
    for bad, err in ((dict(ok, layout="rows"), ValueError), (dict(ok, norm="group"), ValueError),
                     (dict(ok, table=t[:-1]), ValueError), (dict(ok, table=None), TypeError),
                     (dict(ok, axes=(0, 32, 34)), ValueError), (dict(ok, axes=(0, 16, 32)), ValueError),
                     (dict(ok, q_weight=t[:, 0]), ValueError),
                     (dict(ok, norm="head", q_weight=torch.ones(32, device="cuda")), ValueError),
                     (dict(ok, norm="head", q_weight=torch.ones(64)), ValueError),
                     (dict(ok, norm="head", eps=0.0), basa.BasaError),
                     (dict(ok, out_dtype=F32), TypeError), (dict(ok, out=(q[:, :, :2], q, q)), ValueError),
                     (dict(ok, descale=(-1.0, 0.0, 0.0)), basa.BasaError)):
        with pytest.raises(err):
            basa.qkv_rope(q, q, q, **bad)
    with pytest.raises(TypeError):
        basa.qkv_rope(q, q.float(), q, **ok)
    with pytest.raises(ValueError):
        basa.qkv_rope(q[..., ::2], q[..., ::2], None, **ok)
    with pytest.raises(ValueError):
        basa.qkv_rope(q, q[:, :, :, :, :, :32].contiguous(), None, **ok)
    with pytest.raises(ValueError, match="workspace"):
        basa.qkv_rope_bwd(q, q, q, q, q, t, (0, 32, 32), norm="head", q_weight=torch.ones(64, device="cuda"),
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    x = rnd(2, 2, 6, 64, dtype=BF)
    for bad, err in ((dict(norm="batch"), ValueError), (dict(gate=x[:, 0, :32]), ValueError),
                     (dict(gate=x[:1, 0]), ValueError), (dict(scale=x[:, 0], shift=x[0, 0]), ValueError),
                     (dict(gate=x[:, 0], scale=x[:, 0].float()), TypeError), (dict(weight=x[0]), ValueError),
                     (dict(gate=x[:, :4]), ValueError), (dict(eps=-1.0), basa.BasaError),
                     (dict(h_dtype=F32), TypeError), (dict(x_out=x.float()), TypeError),
                     (dict(norm=None, scale=x[:, 0]), basa.BasaError), (dict(norm=None, h_out=x), ValueError),
                     (dict(res_scale=float("nan")), basa.BasaError)):
        with pytest.raises(err):
            basa.gated_norm(x, x, **bad)
    for bad in (dict(gate=x[:, 0]), dict(post_norm="rms"), dict(norm=None), dict(x_out=x), dict(res_scale=2.0)):
        with pytest.raises(ValueError):
            basa.gated_norm(x, None, **bad)
    with pytest.raises(basa.BasaError):
        basa.gated_norm(x, x.float())
    st = torch.zeros(2, 6, 4, device="cuda")
    for a in ((x, x, None, x, x), (None, x, st, x, x), (x, None, st, x, x), (x, x, st[:1], x, x), (x, x, st, x, x[:1])):
        with pytest.raises((ValueError, TypeError)):
            basa.gated_norm_bwd(*a)
    with pytest.raises(ValueError):
        basa.gated_norm(x.transpose(0, 1), x)
    assert basa.get_status() == 0


def test_block_bf16_preparation_feeds_the_attention(basa):
    """qkv_rope's outputs through window_attn, and its gradients through the backward, against the
    oracle on the same values (bf16, and e4m3 with its factors)."""
    shape, window, shift = (1, 1, 32, 32, 2, 128), (1, 16, 16), (0, 8, 8)
    lead, axes = shape[:4], (16, 56, 56)
    table = basa.rope_table((1, 32, 32), axes)
    whole = rnd(3, *lead, 6 * 128, dtype=BF)
    q, k, v = (t.view(*lead, 2, 128) for t in whole.split(256, -1))
    w = rnd(4, 128, dtype=BF, mean=1.0, std=0.1)
    f = oracle.as_f64
    args = dict(norm="head", q_weight=w, k_weight=w)
    qo, ko, vo = basa.qkv_rope(q, k, v, table, axes, **args)
    out, lse = basa.window_attn(qo, ko, vo, window, shift, return_lse=True)
    prm = oracle_params(shape, window, shift)
    assert_close(out, oracle.window_attn(f(qo), f(ko), f(vo), prm), "bf16", "attention of rotated q, k")
    g = rnd(5, *shape, dtype=BF)
    grads = basa.window_attn_bwd(qo, ko, vo, out, g, lse, window, shift)
    refs = oracle.window_attn_bwd(f(qo), f(ko), f(vo), f(g), prm)
    for a, b in zip(grads, refs):
        assert_close(a, b, "bf16", "gradients of rotated q, k")
    dwhole = torch.empty_like(whole)
    into = [t.view(*lead, 2, 128) for t in dwhole.split(256, -1)]
    basa.qkv_rope_bwd(*grads, q, k, table, axes, out=into, **args)
    cs = table64(table, (1, 32, 32), axes)
    for i, (gr, x) in enumerate(zip(grads, (q, k))):
        ref, mag, _, _ = rope_bwd64(gr, x, w, cs, axes, "pairs", "head", 1e-6)
        check(into[i], ref, mag, K_ROW, "gradient through the norm")
    descale = (0.02, 0.02, 0.01)
    q8, k8, v8 = basa.qkv_rope(q, k, v, table, axes, out_dtype=E4, descale=descale, **args)
    out8 = basa.window_attn(q8, k8, v8, window, shift, descale=descale)
    ref = oracle.window_attn(*(f(t) * s for t, s in zip((q8, k8, v8), descale)), prm)
    assert_close(out8, ref, "bf16", "attention of e4m3 q, k")


def test_block_fp32_end_to_end(basa):
    """A block's chain in fp32, forward and backward: border, projection, preparation, window attention,
    projection, border, against autograd in 64 bits.  Five stages of relative error below K_ROW 2^-24 each
    forward and as many backward, amplified by each stage's condition of a few: 2^-24 * 66 * 10 * 4 = 1.6e-4
    at the outermost, relative to the tensor's norm."""
    B, grid, H, d, C = 1, (1, 8, 8), 2, 64, 128
    n, window, shift, axes = 64, (1, 4, 4), (0, 2, 2), (0, 32, 32)
    table = basa.rope_table(grid, axes)
    names = {"x": (B, n, C), "y": (B, n, C), "w1": (C, 3 * C), "w2": (C, C), "gate": (B, C), "scale": (B, C),
             "shift": (B, C), "qw": (d,), "kw": (d,), "pw": (C,)}
    s = {k: rnd(i + 1, *v, std=0.08 if k[0] == "w" else 0.5, mean=1.0 if k in ("qw", "kw", "pw") else 0.0)
         for i, (k, v) in enumerate(names.items())}
    gh, gx = rnd(50, B, n, C), rnd(51, B, n, C)
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        mods = dict(gate=s["gate"], scale=s["scale"], shift=s["shift"], post_weight=s["pw"], post_norm="rms")
        x1, h1, st1 = basa.gated_norm(s["x"], s["y"], return_stats=True, **mods)
        qkv = h1 @ s["w1"]
        q, k, v = (t.view(B, *grid, H, d) for t in qkv.split(C, -1))
        rope = dict(norm="head", q_weight=s["qw"], k_weight=s["kw"])
        qo, ko, vo = basa.qkv_rope(q, k, v, table, axes, **rope)
        o, lse = basa.window_attn(qo, ko, vo, window, shift, return_lse=True)
        y2 = o.view(B, n, C) @ s["w2"]
        x2, h2, st2 = basa.gated_norm(x1, y2, return_stats=True, **mods)
        g2 = basa.gated_norm_bwd(gh, x2, st2, y2, gx, **mods)
        do = (g2.dy @ s["w2"].T).view(B, *grid, H, d)
        dw2 = o.view(n, C).T @ g2.dy.view(n, C)
        dq, dk, dv = basa.window_attn_bwd(qo, ko, vo, o, do, lse, window, shift)
        dqkv = torch.empty_like(qkv)
        into = [t.view(B, *grid, H, d) for t in dqkv.split(C, -1)]
        _, _, _, dqw, dkw = basa.qkv_rope_bwd(dq, dk, dv, q, k, table, axes, out=into, **rope)
        dw1 = h1.view(n, C).T @ dqkv.view(n, 3 * C)
        g1 = basa.gated_norm_bwd(dqkv @ s["w1"].T, x1, st1, s["y"], g2.dx, **mods)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = old
    # 64 bits
    z = {k: t.double().requires_grad_() for k, t in s.items()}
    cs = table64(table, grid, axes)
    ids = torch.tensor([((yy - 2) % 8 // 4) * 2 + (xx - 2) % 8 // 4 for yy in range(8) for xx in range(8)],
                       device="cuda")

    def border(x, y):
        u = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * z["pw"]
        x = x + z["gate"][:, None] * u
        c = x - x.mean(-1, keepdim=True)
        h = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-6)
        return x, h * (1 + z["scale"][:, None]) + z["shift"][:, None]

    def prep(t, w):
        t = t.view(B, *grid, H, d)
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = t[..., 0::2], t[..., 1::2]
        c, sn = cs[..., 0].unsqueeze(3), cs[..., 1].unsqueeze(3)
        return torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2).view(n, H, d).transpose(0, 1)
    r1, rh1 = border(z["x"], z["y"])
    rq, rk, rv = (rh1 @ z["w1"]).split(C, -1)
    rq, rk, rv = prep(rq, z["qw"]), prep(rk, z["kw"]), rv.reshape(n, H, d).transpose(0, 1)
    att = (rq @ rk.transpose(1, 2) / math.sqrt(d)).masked_fill(ids[:, None] != ids[None], float("-inf")).softmax(-1)
    ro = (att @ rv).transpose(0, 1).reshape(B, n, C)
    r2, rh2 = border(r1, ro @ z["w2"])
    ((rh2 * gh.double()).sum() + (r2 * gx.double()).sum()).backward()
    got = {"x": g1.dx, "y": g1.dy, "w1": dw1, "w2": dw2, "gate": g1.dgate + g2.dgate, "scale": g1.dscale + g2.dscale,
           "shift": g1.dshift + g2.dshift, "qw": dqw, "kw": dkw, "pw": g1.dpost_weight + g2.dpost_weight}
    tol = U * K_ROW * 40
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(x2, r2) <= tol and rel(h2, rh2) <= tol
    for name, t in got.items():
        assert rel(t, z[name].grad.view(t.shape)) <= tol, name
