"""The operators around the head in the debug-checks build (no flag, the same bits), at random sizes and layouts
against their 64-bit forms, and at the ends of what they take."""
import math
import random

import pytest
import torch

import training_ref as ref
from test_gpu_training import PAIRS, TYPES, many_tokens, norm_inputs, randn, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    build.build(debug_checks=True)
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def every_call(rlk, T, H, V, dtype, pad, err):
    gen = rng(T + H + V)
    k = dict(err_flag=err)
    table, dout = randn(gen, V, H, dtype=dtype, pad=pad, shift=pad), randn(gen, T, H, dtype=dtype, pad=pad, shift=pad)
    ids = many_tokens(gen, T, V, "zipf")
    o = [rlk.embedding_fwd(table, ids, scale=0.5, **k), rlk.embedding_bwd(dout, ids, V, **k),
         rlk.embedding_bwd(dout, ids, V, out=torch.ones((V, H), device="cuda"), accumulate=True, **k)]
    for centered in (True, False):
        x, w, b, dy = norm_inputs(gen, T, H, dtype, dtype, dtype, pad, pad)
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, centered=centered, **k)
        o += [y, rstd, *rlk.layer_norm_bwd(dy, x, w, mean, rstd, **k)]
    grads = [dout.contiguous(), table.contiguous(), ids.float()]
    out = [torch.empty_like(g) for g in grads]
    return o + [rlk.grad_norm(grads, **k), rlk.clip_grad_norm(grads, 0.3, out=out, **k), *out]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,V,pad", [(1, 1, 1, 0), (7, 65, 30, 1), (300, 520, 700, 0), (300, 1001, 90, 3), (1500, 4096, 300, 8),
                                       (40, 8200, 20, 0), (33, 16400, 8, 1), (5000, 24, 6000, 0)])
def test_checked_build(rlk, dtype, T, H, V, pad):
    from deterministic_token_logprob_gb300 import build
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = every_call(rlk, T, H, V, dtype, pad, err)
    with rlk.library(build.DEBUG_LIB):
        assert rlk.debug_checks()
        checked = every_call(rlk, T, H, V, dtype, pad, err)
    assert int(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(plain, checked))


def test_random_sizes(rlk):
    """Sizes, types, alignments and distances drawn over small ranges, every boundary of the kernels' choices among them."""
    r = random.Random(5)
    edges = [1, 8, 255, 256, 257, 511, 512, 520, 776, 1023, 1024, 1032, 1288, 2040, 2048, 2056, 3000, 4088, 4096, 4104]
    for case in range(120):
        H = r.choice(edges) if r.random() < 0.5 else r.randrange(1, 5000)
        T = r.choice([1, 2, 15, 16, 17, 255, 256, 257, 600]) if r.random() < 0.6 else r.randrange(1, 900)
        dtype, out = r.choice(PAIRS)
        pad, shift = r.choice([(0, 0), (0, 0), (8, 0), (r.randrange(9), r.randrange(9))])
        gen = rng(case)
        if case % 3 == 0:
            V = r.choice([1, 2, 100, 1217, 3000, 5000])
            table = randn(gen, V, H, dtype=dtype, pad=pad, shift=shift)
            ids = many_tokens(gen, T, V, r.choice(["zipf", "even", "runs"]))
            got = rlk.embedding_fwd(table, ids, scale=1.5, out_dtype=out)
            want, tol = ref.lookup(table, ids, 1.5, 0, V)
            ref.close(got, want, ref.rounded(want, out, tol), f"lookup {case}")
            dout = randn(gen, T, H, dtype=dtype, pad=pad, shift=shift)
            want, tol = ref.table_grad(dout, ids, V, 1.5, 0, V, None)
            ref.close(rlk.embedding_bwd(dout, ids, V, scale=1.5), want, tol + ref.TINY[torch.float32], f"table {case}")
            added = torch.full((V, H), 0.25, device="cuda")
            want, tol = ref.table_grad(dout, ids, V, 1.5, 0, V, added)
            ref.close(rlk.embedding_bwd(dout, ids, V, scale=1.5, out=added.clone(), accumulate=True), want, tol, f"added {case}")
        elif case % 3 == 1:
            x, w, b, dy = norm_inputs(gen, T, H, dtype, out, r.choice([dtype, torch.float32]), pad, shift)
            centered = r.random() < 0.5
            y, mean, rstd = rlk.layer_norm_fwd(x, w, b, centered=centered, out_dtype=out)
            (wy, wm, wr), (ty, tm, tr) = ref.norm(x, w, b, 1e-5, centered)
            ref.close(y, wy, ref.rounded(wy, out, ty), f"y {case}")
            ref.close(rstd, wr, tr, f"rstd {case}")
            got = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
            want, tol = ref.norm_grad(dy, x, w, mean, rstd)
            for g, a, t in zip(got, want, tol):
                ref.close(g, a, ref.rounded(a, g.dtype, t), f"norm gradient {case}")
        else:
            sizes = [r.choice([0, 1, 7, 4096, 8191, 8193, r.randrange(1, 60000)]) for _ in range(r.choice([1, 3, 40]))]
            flat = torch.randn(sum(sizes) + shift, generator=gen, device="cuda").to(dtype)[shift:]
            grads = list(flat.split(sizes))
            want, rel = ref.total_norm(grads)
            if not want:
                continue
            to = torch.zeros(sum(sizes) + pad, dtype=out, device="cuda")[pad:]
            norm = rlk.clip_grad_norm(grads, want / 2, out=list(to.split(sizes)))
            assert abs(float(norm) - want) <= rel * want
            exact = flat.double() / 2
            ref.close(to, exact, ref.rounded(exact, out, exact.abs() * (rel + 2 * ref.U)), f"clip {case}")


def test_very_many_tokens(rlk):
    """A token that comes a million times, among three million: runs, groups, and groups of groups."""
    T, H, V = 3_000_001, 2, 1000
    gen = rng(1)
    ids = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.4, 7, torch.randint(0, V, (T,), generator=gen, device="cuda"))
    dout = torch.randn((T, H), generator=gen, device="cuda")
    want, tol = ref.table_grad(dout, ids, V, 1.0, 0, V, None)
    ref.close(rlk.embedding_bwd(dout, ids, V), want, tol)


def test_very_many_gradients(rlk):
    """More tensors than one launch has room for, most of them empty or tiny."""
    gen = rng(2)
    sizes = [(i * 7) % 23 for i in range(5000)] + [100000]
    flat = torch.randn(sum(sizes), generator=gen, device="cuda")
    grads = list(flat.split(sizes))
    want, rel = ref.total_norm([flat])
    n = 0.5 * sum(-(-s * 4 // 16384) for s in sizes) * ref.U     # as many chunks as tensors at most
    norm = rlk.grad_norm(grads)
    assert abs(float(norm) - want) <= (rel + n) * want
    before = flat.clone()
    assert torch.equal(rlk.clip_grad_norm(grads, want / 4), norm)
    exact = before.double() / 4
    ref.close(flat, exact, ref.rounded(exact, torch.float32, exact.abs() * (rel + n + 2 * ref.U)))


def test_narrow_and_wide_ends(rlk):
    """One column, one row, the widest row, the largest vocabulary."""
    x = torch.randn((100000, 1), generator=rng(3), device="cuda")
    y, mean, rstd = rlk.layer_norm_fwd(x)
    assert torch.equal(mean, x[:, 0]) and not y.any()
    dx, dw, db = rlk.layer_norm_bwd(x, x, None, mean, rstd)
    # dx = r (g - mean g): g less itself; dw of h = 0
    assert not dx.any() and not dw.any()
    assert abs(float(db) - float(x.double().sum())) <= 400 * ref.U * float(x.double().abs().sum())
    V = 1 << 24
    table = torch.arange(V, device="cuda", dtype=torch.float32)[:, None]
    ids = torch.tensor([V - 1, 0, V // 2 + 1, -1], device="cuda")
    assert rlk.embedding_fwd(table, ids)[:, 0].tolist() == [float(V - 1), 0.0, float(V // 2 + 1), 0.0]
    for n in (1, 100):
        g = rlk.embedding_bwd(torch.ones((4 * n, 1), device="cuda"), ids.repeat(n), V)
        assert float(g.sum()) == 3.0 * n and g[ids[:3], 0].tolist() == [float(n)] * 3
    w = torch.randn((2, 65536), generator=rng(4), device="cuda")
    y, mean, rstd = rlk.layer_norm_fwd(w)
    assert abs(float(y.double().square().mean()) - 1) < 1e-4 and math.isfinite(float(rstd.sum()))
