"""The calls around the attention (qkv_rope, gated_norm and their backwards) at values, threads and
buffers where they could go wrong: ties of the output's rounding, infinities beside what is not
rotated, rows of another sample, two host threads, workspaces of exactly the size asked for."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def basa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_diffusion_basa_b200 import build
    build.build()
    import sparse_attention_diffusion_basa_b200 as m
    return m


def rnd(seed, *shape, dtype=F32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8)


def equal(a, b):
    """The same bits; None beside None."""
    return (a is None and b is None) or torch.equal(bits(a), bits(b))


def test_scalar_tensors_follow_their_values(basa):
    """Factors held in 0-dim tensors and updated in place, as a running e4m3 scale is."""
    q, k, v = (rnd(i, 1, 1, 4, 8, 2, 64, dtype=BF) for i in range(3))
    x, y = rnd(4, 2, 9, 128, dtype=BF), rnd(5, 2, 9, 128, dtype=BF)
    for where in ("cpu", "cuda"):
        s, r = torch.tensor(0.04, device=where), torch.tensor(1.0, device=where)
        for value, res in ((0.04, 1.0), (0.08, 0.5), (0.02, -2.0)):
            s.fill_(value)
            r.fill_(res)
            got = basa.qkv_rope(q, k, v, norm="head", out_dtype=E4, descale=(s, s, s))
            want = basa.qkv_rope(q, k, v, norm="head", out_dtype=E4, descale=(value,) * 3)
            assert all(equal(a, b) for a, b in zip(got, want))
            got, want = basa.gated_norm(x, y, res_scale=r), basa.gated_norm(x, y, res_scale=res)
            assert all(equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [None, "head", "token"])
def test_e4m3_is_the_rounded_quotient(basa, dtype, norm):
    """v, and q and k without a norm or angles, are value / factor rounded to fp32 and then to e4m3,
    at the values of bf16 where ties lie (0.75 / 0.03 = 25, between 24 and 26).  The oracle divides in
    64 bits: rounding that quotient to 24 bits gives the correctly rounded one, since 53 >= 2 * 24 + 2.
    So every element has to be equal."""
    m = torch.arange(128, 256, dtype=torch.float64) / 128           # every significand of bf16
    vals = torch.cat([s * m * 2.0 ** e for e in range(-12, 5) for s in (1.0, -1.0)])
    x = vals.to(dtype).cuda().view(1, 1, 1, 34, 1, 128)
    for factor in (0.03, 0.04, 0.07, 1.0 / 3.0, 3.0, 0.0):
        f32 = torch.tensor(factor or 1.0, dtype=F32).double()
        want = (vals.to(dtype).double() / f32).float().clamp(-448.0, 448.0).to(E4).view(x.shape)
        got = basa.qkv_rope(x, x, x, norm=norm, out_dtype=E4, descale=(factor,) * 3)
        for name, o in zip("qkv", got):
            if name == "v" or norm is None:
                off = (o.cpu().float() != want.float()).sum().item()
                assert off == 0, f"{name} / {factor}: {off} of {o.numel()} values"
    far = torch.tensor([float("inf"), -float("inf"), 1e30, -1e30, float("nan"), 0.0, -0.0, 1.0]).to(dtype)
    x = far.cuda().repeat(16).view(1, 1, 1, 1, 1, 128)
    for factor in (1e-30, 1e-3, 0.5, 1e30):  # the outermost factors that are taken, nearly
        _, _, v = basa.qkv_rope(x, x, x, norm=norm, out_dtype=E4, descale=(factor,) * 3)
        want = (far.float() / torch.tensor(factor, dtype=F32)).clamp(-448.0, 448.0).to(E4).repeat(16)
        assert equal(v.cpu().view(-1)[:4], want[:4]) and equal(v.cpu().view(-1)[5:8], want[5:8])
        assert torch.isnan(v.cpu().view(-1)[4].float())


@pytest.mark.parametrize("lead,mods", [((2, 1), 1), ((4, 5), 1), ((1, 9), 2), ((3, 7), 2), ((2, 333), 1)])
@pytest.mark.parametrize("C", [256, 5120, 5128])
@pytest.mark.parametrize("post", [None, "layer"])
def test_border_gradients_of_a_clean_sample_stay_clean(basa, lead, mods, C, post):
    """A row that is not finite belongs to one row of modulations: the others' sums, and the rows
    around it, have the bits of a run without it (odd counts, so that a last row stands alone)."""
    x, y, gh, gx = (rnd(i, *lead, C) for i in range(4))
    gate, scale, shift = (rnd(10 + i, *lead[:mods], C) for i in range(3))
    kw = dict(gate=gate, scale=scale, shift=shift, norm="layer", post_norm=post)
    _, _, st = basa.gated_norm(x, y, return_stats=True, **kw)
    clean = basa.gated_norm_bwd(gh, x, st, y, gx, **kw)
    groups = gate.numel() // C
    per = x.numel() // C // groups
    for g in range(groups):
        for value in (float("inf"), float("nan")):
            xb, yb, sb = x.clone().view(-1, C), y.clone().view(-1, C), st.clone().view(-1, 4)
            xb[g * per, 3] = yb[g * per, 5] = value  # its first row
            sb[g * per] = value
            got = basa.gated_norm_bwd(gh, xb.view(x.shape), sb.view(st.shape), yb.view(x.shape), gx, **kw)
            others = [i for i in range(groups) if i != g]
            for name in ("dgate", "dscale", "dshift"):
                a, b = getattr(got, name).view(groups, C)[others], getattr(clean, name).view(groups, C)[others]
                assert equal(a, b), (name, g)
            rows = [i for i in range(groups * per) if i != g * per]
            assert equal(got.dx.view(-1, C)[rows], clean.dx.view(-1, C)[rows])
            assert equal(got.dy.view(-1, C)[rows], clean.dy.view(-1, C)[rows])
        if g == 3:
            break


def tail_case(layout, d, axes, dtype):
    """(grid, rotated elements, an element of the rest and, for pairs, its neighbour)."""
    rot = sum(axes)
    q = rnd(1, 2, 1, 3, 5, 3, d, dtype=dtype)
    return (1, 3, 5), rot, q


TAILS = [("pairs", 64, (0, 14, 10)), ("pairs", 128, (16, 40, 6)), ("pairs", 32, (0, 0, 2)), ("pairs", 64, (0, 0, 0)),
         ("halves", 64, (0, 16, 16)), ("halves", 128, (16, 40, 24)), ("halves", 128, (0, 0, 0))]


@pytest.mark.parametrize("layout,d,axes", TAILS)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (BF, E4), (F32, E4)])
def test_what_is_not_rotated_is_not_touched(basa, layout, d, axes, dtype, out):
    """Without a norm the rest of a head comes through as it is, signs of zeros too, and an infinity
    there changes nothing beside it: forward (e4m3 stores the largest value) and backward."""
    grid, rot, q = tail_case(layout, d, axes, dtype)
    table = basa.rope_table(grid, axes)
    clean, _, _ = basa.qkv_rope(q, q, None, table, axes, layout=layout, out_dtype=out)
    for e in sorted({rot, rot + 1, rot + 4, d - 2, d - 1}):
        bad = q.clone()
        bad[1, 0, 2, 3, 1, e] = float("inf")
        bad[0, 0, 0, 0, 2, e] = float("-inf")
        bad[0, 0, 1, 1, 0, e] = -0.0
        got, gotk, _ = basa.qkv_rope(bad, bad, None, table, axes, layout=layout, out_dtype=out)
        want = clean.clone()
        want[..., rot:] = bad[..., rot:].float().clamp(-448.0, 448.0).to(E4) if out == E4 else bad[..., rot:]
        assert equal(got, want) and equal(gotk, want), e
        if out != E4:
            dq, dk, _, _, _ = basa.qkv_rope_bwd(bad, bad, None, None, None, table, axes, layout=layout)
            back, _, _, _, _ = basa.qkv_rope_bwd(q, q, None, None, None, table, axes, layout=layout)
            back[..., rot:] = bad[..., rot:]
            assert equal(dq, back) and equal(dk, back), e


def raw_calls(basa, C):
    """The four entries that take shared memory by their width, on one row: no-argument functions that
    return the library's code.  What they read and write is kept by them."""
    from sparse_attention_diffusion_basa_b200 import _lib
    lib, stream = _lib.load(), torch.cuda.Stream()
    H = C // 128
    x, y, h, dx, dy, dq, dk = (torch.zeros(1, C, device="cuda") for _ in range(7))
    st, w = torch.ones(1, 4, device="cuda"), torch.ones(C, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    g = _lib.BasaGnormParams(1, 1, C, 1, 0, 1e-6, 1e-6, 1.0, 0, 0, 0, 0, 0, 0, 0)
    r = _lib.BasaRopeParams(1, H, H, 1, 1, 1, 128, 0, 0, 0, 0, 2, 1e-6, 0, 0, 0)
    assert lib.basa_qkv_rope_bwd_workspace_size(ctypes.byref(r)) <= ws.numel()
    p = {k: t.data_ptr() for k, t in dict(x=x, y=y, h=h, dx=dx, dy=dy, dq=dq, dk=dk, st=st, w=w, ws=ws).items()}
    keep = (x, y, h, dx, dy, dq, dk, st, w, ws, stream)
    s, g_, r_ = stream.cuda_stream, ctypes.byref(g), ctypes.byref(r)
    torch.cuda.synchronize()

    def border(_=keep):
        return lib.basa_gated_norm(p["x"], p["y"], None, None, None, None, None, None, p["x"], p["h"], None, g_, s)

    def border_bwd(_=keep):
        return lib.basa_gated_norm_bwd(p["h"], p["x"], p["st"], None, None, None, None, None, None, None, p["dx"],
                                       p["dy"], None, None, None, None, None, None, None, g_, s)

    def prep(_=keep):
        return lib.basa_qkv_rope(p["x"], p["y"], None, p["w"], p["w"], None, p["dx"], p["dy"], None, r_, s)

    def prep_bwd(_=keep):
        return lib.basa_qkv_rope_bwd(p["x"], p["y"], None, p["x"], p["y"], p["w"], p["w"], None, p["dx"], p["dy"],
                                     None, p["dq"], p["dk"], p["ws"], r_, s)
    return dict(border=border, border_bwd=border_bwd, prep=prep, prep_bwd=prep_bwd)


def run_threads(jobs):
    """Each job in a thread of its own, all let go at once; what they raised."""
    failed, start = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            start.wait()
            job()
        except BaseException as e:  # reported by the test's own thread
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


@pytest.mark.parametrize("widths", [(5120, 4096, 5120, 3840), (8192, 6144, 7168, 8064)])
@pytest.mark.parametrize("name", ["border", "border_bwd", "prep", "prep_bwd"])
def test_threads_with_different_widths(basa, name, widths):
    """One kernel's calls from four threads, each of another width and so of other bytes of shared
    memory: none may change what another's launch is allowed."""
    calls = [raw_calls(basa, C)[name] for C in widths]

    def job(call):
        codes = [call() for _ in range(1500)]
        assert not any(codes), f"{sum(map(bool, codes))} of {len(codes)} calls refused"
    failed = run_threads([lambda c=c: job(c) for c in calls])
    torch.cuda.synchronize()
    assert not failed, failed


def test_threads_on_their_own_streams(basa):
    """Whole steps from four threads at once have the bits of a step alone."""
    jobs = []
    for i, C in enumerate((5120, 1024, 8192, 2048)):
        x, y, gate = rnd(i, 64, C), rnd(10 + i, 64, C), rnd(20 + i, C)
        q = rnd(30 + i, 1, 1, 4, 16, C // 128, 128, dtype=BF)
        w = rnd(40 + i, C, dtype=BF, mean=1.0)

        def step(x=x, y=y, gate=gate, q=q, w=w):
            xo, h, st = basa.gated_norm(x, y, gate=gate, return_stats=True)
            g = basa.gated_norm_bwd(h, xo, st, y, gate=gate)
            a = basa.qkv_rope(q, q, q, norm="token", q_weight=w, k_weight=w)
            b = basa.qkv_rope_bwd(*a, q, q, norm="token", q_weight=w, k_weight=w)
            return [t for t in (xo, h, st, *g, *a, *b) if t is not None]
        want = step()

        def job(step=step, want=want):
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got = step()
                torch.cuda.current_stream().synchronize()
                assert all(equal(a, b) for a, b in zip(got, want))
        jobs.append(job)
    torch.cuda.synchronize()
    failed = run_threads(jobs)
    assert not failed, failed


def test_modulations_expanded_as_advised(basa):
    """A gate a sample beside a scale a frame, the gate expanded and made contiguous: the formula,
    and a gradient a frame whose sum over frames is the sample's (fp32 sums of 6 rows each way: 2^-21)."""
    x, y = rnd(1, 2, 12, 256), rnd(2, 2, 12, 256)
    gate, scale = rnd(3, 2, 256), rnd(4, 2, 3, 256)
    wide = gate[:, None].expand(2, 3, 256)
    with pytest.raises(ValueError, match="contiguous"):
        basa.gated_norm(x, y, gate=wide, scale=scale)
    wide = wide.contiguous()
    xo, h, st = basa.gated_norm(x, y, gate=wide, scale=scale, return_stats=True)
    want, _ = basa.gated_norm(x, y, gate=gate)
    assert equal(xo, want)
    gh = rnd(5, 2, 12, 256)
    g = basa.gated_norm_bwd(gh, xo, st, y, gate=wide, scale=scale)
    assert g.dgate.shape == wide.shape
    t = g.dx.double() * y.double()  # res_scale 1: dx is the gradient of the sum
    assert ((g.dgate.double().sum(1) - t.sum(1)).abs() <= 2.0 ** -21 * t.abs().sum(1)).all()


def test_overlapping_outputs_are_refused(basa):
    """Before a launch: nothing is written.  Slices of one buffer, and an input's own place, are taken."""
    q, k, v = (rnd(i, 1, 1, 4, 8, 2, 64, dtype=BF) for i in range(3))
    t, u = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    for out in ((t, t, u), (t, u, t), (k, q, u), (t, u, q), (t, t.view(-1).view_as(q), u)):
        with pytest.raises(basa.BasaError, match="INVALID_ARG"):
            basa.qkv_rope(q, k, v, out=out)
        with pytest.raises(basa.BasaError, match="INVALID_ARG"):
            basa.qkv_rope_bwd(q, k, v, None, None, out=out)
    x, y = q.view(1, 32, 128), k.view(1, 32, 128)
    a = t.view(1, 32, 128)
    for kw in (dict(x_out=a, h_out=a), dict(x_out=y), dict(h_out=x), dict(x_out=x, h_out=x)):
        with pytest.raises(basa.BasaError, match="INVALID_ARG"):
            basa.gated_norm(x, y, **kw)
    torch.cuda.synchronize()
    assert (t == 7.0).all() and (u == 7.0).all()
    whole = torch.empty(1, 1, 4, 8, 6, 64, dtype=BF, device="cuda")
    want = basa.qkv_rope_bwd(q, k, v, None, None)
    got = basa.qkv_rope_bwd(q, k, v, None, None, out=whole.split(2, -2))
    assert all(equal(g, w) for g, w in zip(got, want))
    want, got = basa.gated_norm(x, y), basa.gated_norm(x, y, x_out=x, h_out=y)
    assert got[0] is x and got[1] is y
    assert all(equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("lead", [(2, 0), (0, 3), (0, 0)])
def test_no_tokens_with_a_modulation_each(basa, lead):
    x, m = torch.empty(*lead, 64, device="cuda"), torch.empty(*lead, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    xo, h, st = basa.gated_norm(x, x, gate=m, scale=m, shift=m, weight=w, return_stats=True)
    assert xo.shape == h.shape == x.shape and st.shape == (*lead, 4)
    g = basa.gated_norm_bwd(x, xo, st, x, x, gate=m, scale=m, shift=m, weight=w)
    assert g.dgate.shape == g.dscale.shape == g.dshift.shape == m.shape and (g.dweight == 0).all()


GUARD = 1 << 16


def guarded(n):
    """n bytes of 0xff (NaN to whoever reads them unwritten) and a guard behind them."""
    buf = torch.full((n + GUARD,), 0xff, dtype=torch.uint8, device="cuda")
    buf[n:] = 0xa5
    return buf


@pytest.mark.parametrize("with_v", [True, False])
@pytest.mark.parametrize("norm,grid,H,Hkv,d", [
    ("token", (1, 1, 1), 4, 1, 32), ("token", (2, 9, 31), 12, 1, 128), ("token", (1, 40, 60), 8, 8, 64),
    ("token", (1, 37, 41), 2, 1, 32), ("token", (1, 30, 50), 40, 8, 128), ("token", (1, 9, 11), 128, 2, 128),
    ("head", (1, 1, 1), 3, 1, 64), ("head", (1, 64, 65), 24, 8, 128), ("head", (1, 17, 19), 200, 4, 32)])
def test_preparation_backward_keeps_to_its_workspace(basa, norm, grid, H, Hkv, d, with_v):
    """A workspace of exactly the bytes asked for, unwritten before: nothing behind it is touched,
    and the sums are those of the binding's own call and of 64 bits."""
    lead = (1, *grid)
    q, gq = rnd(1, *lead, H, d, dtype=BF), rnd(2, *lead, H, d, dtype=BF)
    k, gk, gv = (rnd(3 + i, *lead, Hkv, d, dtype=BF) for i in range(3))
    gv = gv if with_v else None
    n = (d, d) if norm == "head" else (H * d, Hkv * d)
    qw, kw = (rnd(7 + i, m, mean=1.0, std=0.3) for i, m in enumerate(n))
    from sparse_attention_diffusion_basa_b200 import _lib
    prm = _lib.BasaRopeParams(1, H, Hkv, *grid, d, 0, 0, 0, 0, _lib.BASA_ROPE_NORM[norm], 1e-6, 1, 1, 0)
    need = _lib.load().basa_qkv_rope_bwd_workspace_size(ctypes.byref(prm))
    assert need > 0
    buf = guarded(need)
    args = (gq, gk, gv, q, k)
    kw_ = dict(norm=norm, q_weight=qw, k_weight=kw)
    got = basa.qkv_rope_bwd(*args, workspace=buf[:need], **kw_)
    torch.cuda.synchronize()
    assert (buf[need:] == 0xa5).all()
    with pytest.raises(ValueError, match="workspace"):
        basa.qkv_rope_bwd(*args, workspace=buf[:need - 1], **kw_)
    assert all(equal(a, b) for a, b in zip(got, basa.qkv_rope_bwd(*args, **kw_)))
    dims = (-1,) if norm == "head" else (-2, -1)
    for x, g, w, dw in ((q, gq, qw, got[3]), (k, gk, kw, got[4])):
        x64, g64 = x.double(), g.double()
        r = 1 / torch.sqrt(x64.square().mean(dims, keepdim=True) + 1e-6)
        t = g64 * x64 * r
        over = (0, 1, 2, 3, 4) if norm == "head" else (0, 1, 2, 3)
        # a thread adds fewer than 64 terms, 128 chains add fewer than 32 rows each and are joined in 12
        # steps; 66 roundings stand around a term
        assert ((dw.double() - t.sum(over).reshape(-1)).abs()
                <= 174 * 2.0 ** -24 * t.abs().sum(over).reshape(-1)).all()


@pytest.mark.parametrize("rows,groups,C", [(1, 1, 8), (5, 5, 264), (333, 3, 1000), (6000, 1, 256), (6000, 3000, 64),
                                           (700, 700, 5120), (77, 7, 8192), (4001, 1, 5128)])
def test_border_backward_keeps_to_its_workspace(basa, rows, groups, C):
    """The same of the border, with more and with fewer modulation rows than CTAs."""
    per = rows // groups
    x, y, gh, gx = (rnd(i, groups, per, C, dtype=BF) for i in range(4))
    mods, w = [rnd(10 + i, groups, C) for i in range(3)], [rnd(20 + i, C, dtype=BF, mean=1.0) for i in range(3)]
    kw = dict(gate=mods[0], scale=mods[1], shift=mods[2], post_weight=w[0], weight=w[1], bias=w[2], norm="layer",
              post_norm="rms")
    _, _, st = basa.gated_norm(x, y, return_stats=True, **kw)
    from sparse_attention_diffusion_basa_b200 import _lib
    prm = _lib.BasaGnormParams(rows, groups, C, 1, 2, 1e-6, 1e-6, 1.0, 1, 1, 0, 1, C, C, C)
    need = _lib.load().basa_gated_norm_bwd_workspace_size(ctypes.byref(prm))
    assert need > 0
    buf = guarded(need)
    got = basa.gated_norm_bwd(gh, x, st, y, gx, workspace=buf[:need], **kw)
    torch.cuda.synchronize()
    assert (buf[need:] == 0xa5).all()
    with pytest.raises(ValueError, match="workspace"):
        basa.gated_norm_bwd(gh, x, st, y, gx, workspace=buf[:need - 1], **kw)
    assert all(equal(a, b) for a, b in zip(got, basa.gated_norm_bwd(gh, x, st, y, gx, **kw)))
    # shift's and bias's gradients are plain sums: a thread adds fewer than 64 rows, 1184 partial rows
    # or fewer are added in 32 chains of 37 and joined in 32; a rounding to bf16 for bias
    t = gh.double()
    assert ((got.dshift.double() - t.sum(1)).abs() <= 136 * 2.0 ** -24 * t.abs().sum(1)).all()
    t = t * (1 + mods[1].double()[:, None])
    ref, tol = t.sum((0, 1)), 140 * 2.0 ** -24 * t.abs().sum((0, 1))
    assert ((got.dbias.double() - ref).abs() <= tol + (ref.abs() + tol) * 2.0 ** -8).all()


@pytest.mark.parametrize("C", [264, 1536, 5120, 8192])
@pytest.mark.parametrize("xt,yt", [(F32, BF), (F32, F32), (BF, BF)])
def test_border_in_place_in_every_type(basa, xt, yt, C):
    """x_out in x's place and h in y's, and the backward's dx in dx_out's (the C entry): the bits of a
    call with outputs of its own, with more rows than are worked on at a time."""
    from sparse_attention_diffusion_basa_b200 import _lib
    x, y = rnd(1, 2, 1501, C, dtype=xt), rnd(2, 2, 1501, C, dtype=yt)
    gate, scale = rnd(3, 2, C), rnd(4, 2, C)
    kw = dict(gate=gate, scale=scale, post_norm="rms")
    xo, h, st = basa.gated_norm(x, y, return_stats=True, **kw)
    xc, yc = x.clone(), y.clone()
    basa.gated_norm(xc, yc, x_out=xc, h_out=yc, **kw)
    assert equal(xc, xo) and equal(yc, h)
    gh, gx = rnd(5, 2, 1501, C, dtype=yt), rnd(6, 2, 1501, C, dtype=xt)
    want = basa.gated_norm_bwd(gh, xo, st, y, gx, **kw)
    t = lambda d: 0 if d == F32 else 1  # noqa: E731
    prm = _lib.BasaGnormParams(3002, 2, C, 1, 2, 1e-6, 1e-6, 1.0, t(xt), t(yt), 0, 0, C, C, 0)
    dy, dgate, dscale = torch.empty_like(y), torch.empty_like(gate), torch.empty_like(scale)
    ws = torch.empty(_lib.load().basa_gated_norm_bwd_workspace_size(ctypes.byref(prm)), dtype=torch.uint8, device="cuda")
    p = lambda a: a.data_ptr()  # noqa: E731
    code = _lib.load().basa_gated_norm_bwd(p(gh), p(xo), p(st), p(y), p(gx), p(gate), None, None, None, p(scale), p(gx),
                                           p(dy), p(dgate), None, None, None, p(dscale), None, p(ws),
                                           ctypes.byref(prm), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    for a, b in ((gx, want.dx), (dy, want.dy), (dgate, want.dgate), (dscale, want.dscale)):
        assert equal(a, b)


@pytest.mark.parametrize("norm,H,Hkv", [(None, 5, 5), ("head", 24, 8), ("token", 12, 3), ("token", 40, 40)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_preparation_in_place_over_many_tokens(basa, norm, H, Hkv, dtype):
    """Every output in its input's place where rows are read ahead of those that are written."""
    grid, axes = (3, 31, 47), (44, 42, 42)
    table = basa.rope_table(grid, axes)
    q, k, v = (rnd(i, 1, *grid, n, 128, dtype=dtype) for i, n in enumerate((H, Hkv, Hkv)))
    want = basa.qkv_rope(q, k, v, table, axes, norm=norm)
    place = [t.clone() for t in (q, k, v)]
    basa.qkv_rope(*place, table, axes, norm=norm, out=place)
    assert all(equal(a, b) for a, b in zip(place, want))
    g = [rnd(5 + i, *t.shape, dtype=dtype) for i, t in enumerate((q, k, v))]
    want = basa.qkv_rope_bwd(*g, q, k, table, axes, norm=norm)
    basa.qkv_rope_bwd(*g, q, k, table, axes, norm=norm, out=g)
    assert all(equal(a, b) for a, b in zip(g, want))
