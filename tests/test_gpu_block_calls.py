"""The calls around the attention (qkv_rope, gated_norm and their backwards) at values, threads and
buffers where they could go wrong: ties of the output's rounding, infinities beside what is not
rotated, rows of another sample, two host threads, workspaces of exactly the size asked for."""
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
