"""The norm's gradient and the gradient norm at the ends of fp32, against 64-bit forms with the bounds of training_ref."""
import math

import pytest
import torch

import training_ref as ref
from test_gpu_training import norm_inputs, randn, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def far_rows(gen, H, dtype):
    """Offsets much larger than what varies, rows near both ends of fp32, and rows that differ from their mean by more than
    fp32 holds (H of one column has none)."""
    z = torch.randn((6, H), generator=gen, device="cuda")
    two = torch.full_like(z[0], 2e38)
    two[::max(8, H // 2)] = -3e38                             # x - m below -2^128
    sides = torch.where(torch.arange(H, device="cuda") % 2 == 0, 3.3e38, -3.3e38)
    sides[H // 2] = -3.3e38
    rows = [z[0] + 1000.0, z[1] * 1e30, z[2].clamp(-3, 3) * 1e38, z[3] * 1e-30, torch.full_like(z[4], 3e38), z[5] * 1e-3 - 64.0,
            two, sides, z[0] * 1e-39, z[1]]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("H", [8, 100, 4096, 8193, 16384, 20000])
def test_norm_gradient_far_values(rlk, dtype, out, H):
    """Rows that the forward takes have a gradient that is finite and within the bounds, from the forward's statistics."""
    gen = rng(H)
    x = far_rows(gen, H, dtype)
    assert bool(x.isfinite().all())
    w = torch.randn(H, generator=gen, device="cuda")
    dy = randn(gen, len(x), H, dtype=out)
    odd = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view(x.shape).copy_(x)
    for centered in (True, False):
        y, mean, rstd = rlk.layer_norm_fwd(x, w, centered=centered, out_dtype=out)
        assert bool(y.isfinite().all()) and bool(rstd.isfinite().all())
        got = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        want, tol = ref.norm_grad(dy, x, w, mean, rstd)
        for g, a, t, name in zip(got, want, tol, ("dx", "dw", "db")):
            # a term below fp32's normal values is off by half of the smallest one, the sum by that for each row
            ref.close(g, a, ref.rounded(a, g.dtype, t) + len(x) * ref.TINY[torch.float32], name)
        again = rlk.layer_norm_bwd(dy, odd, w, mean, rstd)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_norm_of_infinities(rlk):
    """The root of a sum with an infinity in it is infinite, and NaN where there is a NaN; a norm beyond fp32 is infinite too."""
    big = torch.finfo(torch.float32).max
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        z = torch.randn(20000, generator=rng(1), device="cuda").to(dtype)
        for at in ([0], [19999], [5, 17000], list(range(0, 20000, 7))):
            for sign in (1, -1):
                g = z.clone()
                g[at] = sign * math.inf
                err = torch.zeros(1, dtype=torch.int32, device="cuda")
                assert float(rlk.grad_norm([z, g], err_flag=err)) == math.inf and int(err) == rlk.RLK_FLAG_NONFINITE
                mine = [z.clone(), g.clone()]
                assert float(rlk.clip_grad_norm(mine, 1.0, err_flag=err)) == math.inf
                assert torch.equal(mine[0], z) and torch.equal(mine[1], g)
                g[1234] = math.nan
                assert math.isnan(float(rlk.grad_norm([g, z])))
    for n in (2, 5000, 3_000_000):
        assert float(rlk.grad_norm(torch.full((n,), big, device="cuda"))) == math.inf
    assert float(rlk.grad_norm(torch.full((1,), big, device="cuda"))) == big


@pytest.mark.parametrize("v", [1e-15, 1.7e-15, 3.3e-16, 1e25, 1.3e25, 1e30])
def test_norm_of_many_elements_far_from_one(rlk, v):
    """2^31 equal elements whose squares are summed at another scale (a power of two, which rounds nothing), 575 chunks a thread. Relative
    to the sum of squares: 9 roundings of a chunk's 16 values, 2 of the sum of chunks, whose losses are kept, 8 in a warp and
    between warps, as many where the shares are joined (3 sums with their losses, 8), and one beside the other scales: 31 half steps
    at most, of which the root leaves 15.5, its own rounding and that of the result's scale apart."""
    g = torch.full((1 << 31,), v, device="cuda")
    want = math.sqrt(2.0 ** 31) * float(g[0])
    assert abs(float(rlk.grad_norm([g])) / want - 1) <= 18 * ref.U


@pytest.mark.parametrize("dtype,out", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("size,max_norm", [(1e36, 1.0), (1e36, 1e-3), (1e35, 1e-9), (1e36, 1e-30), (1e30, 1e-12), (1e36, 2.0 ** -126),
                                           (1e34, 1e-42), (1e5, 1e-40), (1.0, 1e-50), (1e36, 1e30)])
def test_clip_by_factors_below_normal_values(rlk, dtype, out, size, max_norm):
    """max_norm / norm may lie below fp32's normal values where results do not. The factor costs the norm's bound and three half steps
    (the norm's own, max_norm's and the division's), the product two; below the normal values, where the gradient times 2^-126, the norm times
    2^-126 and the factor may lie, half of the smallest value each, times 4 (what a gradient times 2^-126 is at most)."""
    z = torch.randn(30011, generator=rng(4), device="cuda")
    z[::5] *= 1e-6
    flat = (z * size).to(dtype)
    grads = list(flat.split([7, 20000, 10004]))
    want, rel = ref.total_norm(grads)
    f = max_norm / want
    to = torch.full((30011 + 3,), 7.0, dtype=out, device="cuda")
    norm = rlk.clip_grad_norm(grads, max_norm, out=list(to[1:-2].split([7, 20000, 10004])))
    assert abs(float(norm) / want - 1) <= rel
    exact = flat.double() * f
    tol = exact.abs() * (rel + 5 * ref.U) + 8 * ref.TINY[torch.float32]
    ref.close(to[1:-2], exact, ref.rounded(exact, out, tol))
    assert to[0] == 7.0 and to[-2:].tolist() == [7.0, 7.0]
    if dtype is out:
        mine = flat.clone()
        assert torch.equal(rlk.clip_grad_norm(list(mine.split([7, 20000, 10004])), max_norm), norm) and torch.equal(mine, to[1:-2])


def test_clip_many_chunks_by_a_factor_below_normal_values(rlk):
    """The same where a CTA scales one chunk: 2^25 elements of two values, in place."""
    g = torch.full((1 << 25,), 1e34, device="cuda")
    g[::3] = -3e30
    want, _ = ref.total_norm([g])
    exact = g.double() * (1e-5 / want)
    rlk.clip_grad_norm([g], 1e-5)
    # sums of equal squares, 2^25 of them: 40 half steps at most (test_norm_of_many_elements)
    ref.close(g, exact, ref.rounded(exact, torch.float32, exact.abs() * 45 * ref.U))


def test_clip_to_almost_nothing(rlk):
    """A factor that rounds to nothing leaves zeros with the gradients' signs."""
    for max_norm in (1e-45, 1e-50, 1e-300):
        for size in (1e36, 1e5, 1e-3):
            g = (torch.randn(5003, generator=rng(3), device="cuda")[1:] * size)
            sign = g.signbit()
            rlk.clip_grad_norm(g, max_norm)
            assert torch.equal(g.signbit(), sign) and float(g.abs().max()) <= 2.0 ** -149
