"""Cases and plain forms of the operators around shifted window attention.

Two operators, each forward and backward:

* ``qkv_rope``: what turns the rows of a q/k/v projection into the inputs of
  the attention calls.  RMS norm of q and k (over each head, or over all heads
  of a token), then rotary positions with three axes (time, rows, columns), and
  v copied along when the three are slices of one projection output.
* ``gated_norm``: what stands between two blocks of a Diffusion Transformer.
  The branch's output, through its own norm if it has one, is multiplied by the
  gate and added to the (scaled) residual stream; the sum is normalised and
  modulated for the next block.

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, through the public calls of this package.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, way, B, grid, H, Hkv, d, axes, norm, layout="pairs", dtype="bf16", out="", fused=True,
          with_v=True, fresh=False):
    c = {"op": "rope", "way": way, "B": B, "T": grid[0], "Hg": grid[1], "Wg": grid[2], "H": H, "Hkv": Hkv,
         "d": d, "at": axes[0], "ah": axes[1], "aw": axes[2], "norm": norm, "layout": layout, "dtype": dtype,
         "out": out or dtype, "fused": fused, "with_v": with_v, "fresh": fresh}
    return dict(c, name=name) if name else c


def _gnorm(name, way, B, grid, C, norm="layer", post="none", gate=True, mod=True, affine=False, dtype="bf16",
           stream="bf16", frames=False, stats=False):
    c = {"op": "gnorm", "way": way, "B": B, "T": grid[0], "Hg": grid[1], "Wg": grid[2], "C": C, "norm": norm,
         "post": post, "gate": gate, "mod": mod, "affine": affine, "dtype": dtype, "stream": stream,
         "frames": frames, "stats": stats}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest correctness grid: fp32, the pair of an element half a head away
        _rope("rope grid16 f32", "fwd", 1, (1, 16, 16), 2, 2, 64, (0, 32, 32), "head", layout="halves",
              dtype="f32", fused=False),
        # the text stream of a joint block, one sampling step: positions along one axis, made in the call
        _rope("rope text512", "fwd", 1, (1, 1, 512), 24, 24, 128, (0, 0, 128), "head", fresh=True),
        # the image stream of a 2048^2 block: q, k, v are slices of the projection's output
        _rope("rope flux2048", "fwd", 1, (1, 128, 128), 24, 24, 128, (16, 56, 56), "head"),
        # e4m3 attention inputs straight from the projection, grid of an odd aspect
        _rope("rope 45x80 to e4m3", "fwd", 1, (1, 45, 80), 24, 8, 128, (16, 56, 56), "head", out="e4m3"),
        # a video block: one norm over all heads of a token, separate q and k projections
        _rope("rope wan_video", "fwd", 1, (21, 45, 80), 40, 40, 128, (44, 42, 42), "token", fused=False,
              with_v=False),
        # training of a batch of 2048^2 images, gradient written in the projection's layout
        _rope("rope backward flux2048 b2", "bwd", 2, (1, 128, 128), 24, 24, 128, (16, 56, 56), "head"),
        # training on a ragged clip, norm over all heads, grouped K/V heads
        _rope("rope backward clip", "bwd", 2, (13, 18, 31), 12, 4, 128, (44, 42, 42), "token"),
        # text stream between two blocks, one sampling step
        _gnorm("border text512", "fwd", 1, (1, 1, 512), 2048),
        # video block with an fp32 residual stream
        _gnorm("border wan_video", "fwd", 1, (21, 45, 80), 5120, stream="f32"),
        # norms on both sides of the branch, a modulation of its own for every frame, training forward
        _gnorm("border clip sandwich", "fwd", 2, (13, 18, 31), 1536, norm="rms", post="rms", affine=True,
               frames=True, stats=True),
        # training at 16384 tokens and the width of the video model
        _gnorm("border backward 128x128", "bwd", 1, (1, 128, 128), 5120),
        # odd sizes, fp32, every parameter has a gradient
        _gnorm("border backward odd f32", "bwd", 3, (1, 9, 37), 1000, post="rms", affine=True, dtype="f32",
               stream="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    way = rng.choice(["fwd", "bwd"])
    B = rng.choice([1, 1, 2, 3])
    while True:
        if rng.random() < 0.4:
            grid = (1, 1, _log(rng, 1, 2000))
        elif rng.random() < 0.6:
            grid = (1, _log(rng, 3, 150), _log(rng, 3, 150))
        else:
            grid = (_log(rng, 2, 24), _log(rng, 3, 60), _log(rng, 3, 90))
        n = B * grid[0] * grid[1] * grid[2]
        if rng.random() < 0.5:
            d = rng.choice([32, 64, 128, 128])
            Hkv = rng.choice([1, 2, 3, 5, 8, 12, 24])
            H = Hkv * rng.choice([1, 1, 1, 2, 3])
            layout = rng.choice(["pairs", "halves"])
            left = d // 2
            a = [0, 0, 0]
            if grid[0] > 1:
                a[0] = rng.randint(1, left // 2)
            if grid[1] > 1:
                a[1] = rng.randint(1, (left - a[0]) // 2)
            a[2] = left - a[0] - a[1]
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            out = "e4m3" if way == "fwd" and rng.random() < 0.15 else dtype
            fused = rng.random() < 0.6
            if n * (H + 2 * Hkv) * d * (4 if dtype == "f32" else 2) > 400e6:
                continue
            return _rope("", way, B, grid, H, Hkv, d, [2 * x for x in a], rng.choice(["none", "head", "head", "token"]),
                         layout, dtype, out, fused, fused, way == "fwd" and rng.random() < 0.3)
        C = 8 * _log(rng, 8, 1024)
        stream, dtype = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        if n * C > 120e6:
            continue
        post = rng.choice(["none", "none", "rms", "layer"])
        mod = rng.random() < 0.7
        return _gnorm("", way, B, grid, C, rng.choice(["layer", "layer", "rms"]), post, rng.random() < 0.8, mod,
                      rng.random() < 0.4, dtype, stream, grid[0] > 1 and rng.random() < 0.5,
                      way == "fwd" and rng.random() < 0.5)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
EPS = 1e-6
THETA = 10000.0
DESCALE = (0.04, 0.04, 0.03)  # of e4m3 outputs: values of a few units spread over the type's range


def _positions(c):
    # a later chunk of a clip, image axes centred: positions a sampler has in earnest
    start = (7.0 if c["T"] > 1 else 0.0, -0.5 * (c["Hg"] - 1) if c["Hg"] > 1 else 0.0, 0.0)
    return start, (1.0, 1.0, 0.5 if c["Wg"] > 100 else 1.0)


def _table(c, dev):
    """The (cos, sin) pairs of every coordinate: time, then rows, then columns."""
    start, step = _positions(c)
    parts = []
    for G, a, s, e in zip((c["T"], c["Hg"], c["Wg"]), (c["at"], c["ah"], c["aw"]), start, step):
        if a:
            f = THETA ** (-torch.arange(0, a, 2, dtype=torch.float64, device=dev) / a)
            ang = (s + e * torch.arange(G, dtype=torch.float64, device=dev))[:, None] * f
            parts.append(torch.stack([ang.cos(), ang.sin()], -1).reshape(-1, 2))
    return torch.cat(parts).float().contiguous()


def _split(c, x):
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    lead = x.shape[:-1]
    q, k, v = x.split([H * d, Hkv * d, Hkv * d], -1)
    return q.view(*lead, H, d), k.view(*lead, Hkv, d), v.view(*lead, Hkv, d)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = _DT[c["dtype"]]

    def rnd(*shape, mean=0.0, std=1.0, dtype=dt):
        x = torch.empty(shape, dtype=dtype if dtype != torch.float64 else torch.float32, device=dev)
        return x.normal_(mean, std, generator=g)

    lead = (c["B"], c["T"], c["Hg"], c["Wg"])
    s = {"case": c}
    if c["op"] == "rope":
        H, Hkv, d = c["H"], c["Hkv"], c["d"]
        if c["fused"]:
            s["qkv"] = rnd(*lead, (H + 2 * Hkv) * d, std=1.5)
            s["q"], s["k"], s["v"] = _split(c, s["qkv"])
        else:
            s["q"], s["k"] = rnd(*lead, H, d, std=1.5), rnd(*lead, Hkv, d, std=1.5)
            s["v"] = rnd(*lead, Hkv, d) if c["with_v"] else None
        if c["norm"] != "none":
            n = (d, d) if c["norm"] == "head" else (H * d, Hkv * d)
            s["qw"], s["kw"] = (rnd(m, mean=1.0, std=0.2) for m in n)
        else:
            s["qw"] = s["kw"] = None
        s["table"] = None if c["fresh"] else _table(c, dev)
        if c["way"] == "bwd":
            s["gq"], s["gk"] = rnd(*lead, H, d), rnd(*lead, Hkv, d)
            s["gv"] = rnd(*lead, Hkv, d) if c["with_v"] else None
        return s
    C = c["C"]
    st = _DT[c["stream"]]
    chan = 1.0 + 2.0 * torch.rand(C, device=dev, generator=g)  # channels of unlike sizes
    x = (torch.randn(*lead, C, device=dev, generator=g) * chan + 0.3).to(st)
    y = rnd(*lead, C)
    m = (c["B"], c["T"], C) if c["frames"] else (c["B"], C)
    if c["gate"] or c["mod"]:  # slices of the modulation layer's output: gate, shift, scale
        mods = rnd(*m[:-1], 3 * C, std=0.4)
        gate, shift, scale = mods.split(C, -1)
    s.update(x=x, y=y, gate=gate if c["gate"] else None, shift=shift if c["mod"] else None,
             scale=scale if c["mod"] else None)
    s["w"], s["b"] = (rnd(C, mean=1.0, std=0.2), rnd(C, std=0.2)) if c["affine"] else (None, None)
    if c["norm"] == "rms":
        s["b"] = None
    s["pw"] = rnd(C, mean=1.0, std=0.2) if c["affine"] and c["post"] != "none" else None
    if c["way"] == "bwd":  # x stands for the stored sum; its statistics as the forward call leaves them
        s["gh"], s["gx"] = rnd(*lead, C), rnd(*lead, C, dtype=st)
        zero = torch.zeros(lead, device=dev)
        pre = _stats(x.float(), c["norm"])
        post = _stats(y.float(), c["post"]) if c["post"] != "none" else (zero, zero)
        s["stats"] = torch.stack([*pre, *post], -1).contiguous()
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _angles(c, table):
    """cos and sin [T, Hg, Wg, 1, pairs] of every token."""
    T, Hg, Wg = c["T"], c["Hg"], c["Wg"]
    nt, nh, nw = c["at"] // 2, c["ah"] // 2, c["aw"] // 2
    t, h, w = table.split([T * nt, Hg * nh, Wg * nw])
    full = torch.cat([t.view(T, 1, 1, nt, 2).expand(T, Hg, Wg, nt, 2), h.view(1, Hg, 1, nh, 2).expand(T, Hg, Wg, nh, 2),
                      w.view(1, 1, Wg, nw, 2).expand(T, Hg, Wg, nw, 2)], 3)
    return full[..., None, :, 0], full[..., None, :, 1]


def _rotate(c, x, cos, sin):
    p = cos.shape[-1]
    if c["layout"] == "pairs":
        a, b = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
        return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), x[..., 2 * p:]], -1)
    a, b = x[..., :p], x[..., p:2 * p]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., 2 * p:]], -1)


def _rms(c, x):
    """1 / rms of each head, or of all heads of each token."""
    dims = (-1,) if c["norm"] == "head" else (-2, -1)
    return torch.rsqrt((x * x).mean(dims, keepdim=True) + EPS)


def _weight(c, w, heads):
    w = w.float()
    return w if c["norm"] == "head" else w.view(heads, c["d"])


def _to_out(c, x, i):
    if c["out"] == "e4m3":
        return (x / DESCALE[i]).clamp(-448.0, 448.0).to(_DT["e4m3"])
    return x.to(_DT[c["out"]])


def _plain_rope(s):
    c = s["case"]
    table = _table(c, s["q"].device) if c["fresh"] else s["table"]
    cos, sin = _angles(c, table)
    if c["way"] == "fwd":
        outs = []
        for i, (x, w) in enumerate(((s["q"], s["qw"]), (s["k"], s["kw"]))):
            x = x.float()
            if c["norm"] != "none":
                x = x * _rms(c, x) * _weight(c, w, x.shape[-2])
            outs.append(_to_out(c, _rotate(c, x, cos, sin), i))
        if s["v"] is not None:
            outs.append(_to_out(c, s["v"].float(), 2))
        return outs
    grads, weights = [], []
    for g, x, w in ((s["gq"], s["q"], s["qw"]), (s["gk"], s["k"], s["kw"])):
        g = _rotate(c, g.float(), cos, -sin)
        if c["norm"] != "none":
            x = x.float()
            r, wf = _rms(c, x), _weight(c, w, x.shape[-2])
            gw = g * wf
            dims = (-1,) if c["norm"] == "head" else (-2, -1)
            weights.append((g * x * r).sum((0, 1, 2, 3, 4) if c["norm"] == "head" else (0, 1, 2, 3)).reshape(-1).to(w.dtype))
            g = r * (gw - x * (r * r) * (gw * x).mean(dims, keepdim=True))
        grads.append(g.to(_DT[c["dtype"]]))
    if s["gv"] is not None:
        grads.append(s["gv"])
    if c["fused"]:
        grads = [torch.cat([x.flatten(-2) for x in grads], -1)]
    return grads + weights


def _stats(x, kind):
    """(mean, 1 / deviation) over the last axis."""
    mean = x.mean(-1) if kind == "layer" else torch.zeros_like(x[..., 0])
    d = x - mean[..., None]
    return mean, torch.rsqrt((d * d).mean(-1) + EPS)


def _rows(m, x):
    """A modulation [B, C] or [B, T, C] beside the tokens of x."""
    return m.float().view(*m.shape[:-1], *([1] * (x.dim() - m.dim())), m.shape[-1])


def _over_tokens(v, m):
    """Sum over the tokens that share a row of the modulation m."""
    return v.sum(tuple(range(m.dim() - 1, v.dim() - 1)))


def _plain_gnorm(s):
    c = s["case"]
    one = lambda m, x: _rows(m, x) if m is not None else None  # noqa: E731
    if c["way"] == "fwd":
        y = s["y"].float()
        post = (torch.zeros_like(y[..., 0]),) * 2
        if c["post"] != "none":
            post = _stats(y, c["post"])
            y = (y - post[0][..., None]) * post[1][..., None]
            if s["pw"] is not None:
                y = y * s["pw"].float()
        if s["gate"] is not None:
            y = y * _rows(s["gate"], y)
        x = s["x"].float() + y
        pre = _stats(x, c["norm"])
        h = (x - pre[0][..., None]) * pre[1][..., None]
        if s["w"] is not None:
            h = h * s["w"].float()
        if s["b"] is not None:
            h = h + s["b"].float()
        if s["scale"] is not None:
            h = h * (1.0 + _rows(s["scale"], h)) + _rows(s["shift"], h)
        out = [x.to(s["x"].dtype), h.to(s["y"].dtype)]
        return out + [torch.stack([*pre, *post], -1)] if c["stats"] else out
    st = s["stats"]
    gh, x = s["gh"].float(), s["x"].float()
    xh = (x - st[..., 0:1]) * st[..., 1:2]
    scale = one(s["scale"], x)
    m = gh * (1.0 + scale) if scale is not None else gh
    a = m * s["w"].float() if s["w"] is not None else m
    t = a - xh * (a * xh).mean(-1, keepdim=True)
    if c["norm"] == "layer":
        t = t - a.mean(-1, keepdim=True)
    gx = s["gx"].float() + st[..., 1:2] * t
    out = {"dx": gx.to(s["x"].dtype)}
    if s["w"] is not None:
        out["dw"] = (m * xh).sum((0, 1, 2, 3)).to(s["w"].dtype)
    if s["b"] is not None:
        out["db"] = m.sum((0, 1, 2, 3)).to(s["b"].dtype)
    if scale is not None:
        aff = xh * s["w"].float() if s["w"] is not None else xh
        aff = aff + s["b"].float() if s["b"] is not None else aff
        out["dscale"] = _over_tokens(gh * aff, s["scale"]).to(s["scale"].dtype)
        out["dshift"] = _over_tokens(gh, s["shift"]).to(s["shift"].dtype)
    y = s["y"].float()
    e = gx
    if s["gate"] is not None:
        e = e * _rows(s["gate"], e)
    u = y
    if c["post"] != "none":
        yh = (y - st[..., 2:3]) * st[..., 3:4]
        u = yh
        if s["pw"] is not None:
            u = yh * s["pw"].float()
            out["dpw"] = (e * yh).sum((0, 1, 2, 3)).to(s["pw"].dtype)
            e = e * s["pw"].float()
        t = e - yh * (e * yh).mean(-1, keepdim=True)
        if c["post"] == "layer":
            t = t - e.mean(-1, keepdim=True)
        e = t * st[..., 3:4]
    if s["gate"] is not None:
        out["dgate"] = _over_tokens(gx * u, s["gate"]).to(s["gate"].dtype)
    out["dy"] = e.to(s["y"].dtype)
    return out


# ---------------------------------------------------------------------------
# The package's calls
# ---------------------------------------------------------------------------
def _own_rope(s):
    import sparse_attention_diffusion_basa_b200 as basa
    c = s["case"]
    axes, norm = (c["at"], c["ah"], c["aw"]), None if c["norm"] == "none" else c["norm"]
    table = s["table"]
    if c["fresh"]:
        start, step = _positions(c)
        table = basa.rope_table((c["T"], c["Hg"], c["Wg"]), axes, THETA, start, step, device=s["q"].device)
    if c["way"] == "fwd":
        low = c["out"] == "e4m3"
        out = basa.qkv_rope(s["q"], s["k"], s["v"], table, axes, layout=c["layout"], norm=norm, q_weight=s["qw"],
                            k_weight=s["kw"], eps=EPS, out_dtype=_DT["e4m3"] if low else None,
                            descale=DESCALE if low else (0.0, 0.0, 0.0))
        return [x for x in out if x is not None]
    into = None
    if c["fused"]:
        whole = torch.empty_like(s["qkv"])
        into = _split(c, whole)
    dq, dk, dv, dqw, dkw = basa.qkv_rope_bwd(s["gq"], s["gk"], s["gv"], s["q"], s["k"], table, axes,
                                             layout=c["layout"], norm=norm, q_weight=s["qw"], k_weight=s["kw"],
                                             eps=EPS, out=into)
    return [x for x in ([whole] if c["fused"] else [dq, dk, dv]) + [dqw, dkw] if x is not None]


def _own_gnorm(s):
    import sparse_attention_diffusion_basa_b200 as basa
    c = s["case"]
    kw = dict(gate=s["gate"], post_weight=s["pw"], weight=s["w"], bias=s["b"], scale=s["scale"], shift=s["shift"],
              norm=c["norm"], post_norm=None if c["post"] == "none" else c["post"])
    if c["way"] == "fwd":
        return basa.gated_norm(s["x"], s["y"], eps=EPS, return_stats=c["stats"], **kw)
    g = basa.gated_norm_bwd(s["gh"], s["x"], s["stats"], s["y"], s["gx"], **kw)
    out = {"dx": g.dx, "dw": g.dweight, "db": g.dbias, "dscale": g.dscale, "dshift": g.dshift,
           "dpw": g.dpost_weight, "dgate": g.dgate, "dy": g.dy}
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    if own:
        return _own_rope(state) if state["case"]["op"] == "rope" else _own_gnorm(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_gnorm(state)


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    n = c["B"] * c["T"] * c["Hg"] * c["Wg"]
    es = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["op"] == "rope":
        qk, v = n * (c["H"] + c["Hkv"]) * c["d"], n * c["Hkv"] * c["d"] if c["with_v"] else 0
        wide = 0 if c["norm"] == "none" else c["d"] * (2 if c["norm"] == "head" else c["H"] + c["Hkv"])
        if c["way"] == "fwd":
            return {"bytes": (qk + v) * (es[c["dtype"]] + es[c["out"]]) + wide * es[c["dtype"]],
                    "flops": qk * (7 if c["norm"] != "none" else 3)}
        reads = 2 * qk if c["norm"] != "none" else qk
        return {"bytes": (reads + qk + 2 * v + 2 * wide) * es[c["dtype"]],
                "flops": qk * (14 if c["norm"] != "none" else 3)}
    e, r = es[c["dtype"]], es[c["stream"]]
    C, groups = c["C"], c["B"] * (c["T"] if c["frames"] else 1)
    small = (groups * ((1 if c["gate"] else 0) + (2 if c["mod"] else 0)) + (3 if c["affine"] else 0)) * C * e
    stats = 16 * n if c["stats"] or c["way"] == "bwd" else 0
    if c["way"] == "fwd":
        return {"bytes": n * C * (2 * r + 2 * e) + small + stats, "flops": n * C * 14}
    return {"bytes": n * C * (3 * r + 3 * e) + 2 * small + stats, "flops": n * C * 28}


# ---------------------------------------------------------------------------
# From the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(c, x):
    """Rotary positions as a product of complex numbers, angles from the positions themselves."""
    dev, start_step = x.device, _positions(c)
    B, T, Hg, Wg, heads, d = x.shape
    pieces = []
    for i, (G, a) in enumerate(zip((T, Hg, Wg), (c["at"], c["ah"], c["aw"]))):
        j = torch.arange(a // 2, dtype=torch.float64, device=dev)
        pos = start_step[0][i] + start_step[1][i] * torch.arange(G, dtype=torch.float64, device=dev)
        ang = torch.outer(pos, torch.exp(-math.log(THETA) * 2.0 * j / max(a, 1)))
        shape = [1, 1, 1, a // 2]
        shape[i] = G
        pieces.append(ang.view(shape).expand(T, Hg, Wg, a // 2))
    ang = torch.cat(pieces, -1).unsqueeze(3)
    turn = torch.polar(torch.ones_like(ang), ang)
    p = turn.shape[-1]
    rot, rest = x[..., :2 * p], x[..., 2 * p:]
    if c["layout"] == "halves":
        rot = rot.unflatten(-1, (2, p)).transpose(-1, -2).flatten(-2)
    z = torch.view_as_complex(rot.unflatten(-1, (p, 2)).contiguous()) * turn
    rot = torch.view_as_real(z).flatten(-2)
    if c["layout"] == "halves":
        rot = rot.unflatten(-1, (p, 2)).transpose(-1, -2).flatten(-2)
    return torch.cat([rot, rest], -1) if rest.shape[-1] else rot


def _exact_prep(c, x, w):
    if c["norm"] == "head":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    elif c["norm"] == "token":
        flat = x.flatten(-2)
        x = (flat / torch.sqrt(flat.square().mean(-1, keepdim=True) + EPS) * w).view(x.shape)
    return _exact_turn(c, x)


def _exact_rope(c, s):
    f = lambda t: None if t is None else t.double()  # noqa: E731
    if c["way"] == "fwd":
        out = []
        for i, (x, w) in enumerate(((s["q"], s["qw"]), (s["k"], s["kw"]))):
            o = _exact_prep(c, f(x), f(w))
            out.append(o / DESCALE[i] if c["out"] == "e4m3" else o)
        if s["v"] is not None:
            out.append(f(s["v"]) / DESCALE[2] if c["out"] == "e4m3" else f(s["v"]))
        return out
    grads, weights = [], []
    for g, x, w in ((s["gq"], s["q"], s["qw"]), (s["gk"], s["k"], s["kw"])):
        leaf = f(x).requires_grad_()
        wl = f(w).requires_grad_() if w is not None else None
        with torch.enable_grad():
            got = torch.autograd.grad(_exact_prep(c, leaf, wl), [leaf] if wl is None else [leaf, wl], f(g))
        grads.append(got[0])
        weights += got[1:]
    if s["gv"] is not None:
        grads.append(f(s["gv"]))
    if c["fused"]:
        grads = [torch.cat([x.flatten(-2) for x in grads], -1)]
    return grads + weights


def _exact_gnorm(c, s):
    f = lambda t: None if t is None else t.double()  # noqa: E731

    def normed(x, kind):
        if kind == "layer":
            x = x - x.mean(-1, keepdim=True)
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)

    def beside(m, n):  # a row of m for every token
        m = m.reshape(-1, m.shape[-1])
        return m.repeat_interleave(n // m.shape[0], 0)

    C = c["C"]
    n = s["x"].numel() // C

    def branch(y, gate, pw):
        u = normed(y, c["post"]) if c["post"] != "none" else y
        u = u * pw if pw is not None else u
        return u * beside(gate, n) if gate is not None else u

    def border(x, w, b, scale, shift):
        h = normed(x, c["norm"])
        h = h * w if w is not None else h
        h = h + b if b is not None else h
        return h * (1 + beside(scale, n)) + beside(shift, n) if scale is not None else h

    x, y = f(s["x"]).view(n, C), f(s["y"]).view(n, C)
    if c["way"] == "fwd":
        xo = x + branch(y, f(s["gate"]), f(s["pw"]))
        out = [xo.view(s["x"].shape), border(xo, f(s["w"]), f(s["b"]), f(s["scale"]), f(s["shift"])).view(s["x"].shape)]
        if c["stats"]:
            def two(v, kind):
                mean = v.mean(-1) if kind == "layer" else torch.zeros_like(v[:, 0])
                return [mean, 1 / torch.sqrt((v - mean[:, None]).square().mean(-1) + EPS)]
            post = two(y, c["post"]) if c["post"] != "none" else [torch.zeros_like(x[:, 0])] * 2
            out.append(torch.stack(two(xo, c["norm"]) + post, -1).view(*s["x"].shape[:-1], 4))
        return out
    names = {"w": s["w"], "b": s["b"], "scale": s["scale"], "shift": s["shift"]}
    leaves = {k: f(v).requires_grad_() for k, v in names.items() if v is not None}
    x.requires_grad_()
    with torch.enable_grad():
        h = border(x, *(leaves.get(k) for k in ("w", "b", "scale", "shift")))
        got = torch.autograd.grad(h, [x, *leaves.values()], f(s["gh"]).view(n, C))
    del h
    dx = got[0] + f(s["gx"]).view(n, C)
    out = {"dx": dx.view(s["x"].shape)}
    out.update({"d" + k: v for k, v in zip(leaves, got[1:])})
    two = {k: f(s[k]).requires_grad_() for k in ("gate", "pw") if s[k] is not None}
    y.requires_grad_()
    with torch.enable_grad():
        u = branch(y, two.get("gate"), two.get("pw"))
        got = torch.autograd.grad(u, [y, *two.values()], dx)
    out["dy"] = got[0].view(s["y"].shape)
    out.update({"d" + k: v for k, v in zip(two, got[1:])})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_gnorm(case, s)
