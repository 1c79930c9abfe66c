"""The operators around the head against their 64-bit forms, at the sizes, types, layouts and values
where they can go wrong; bounds are derived in training_ref.py."""
import math

import pytest
import torch

import training_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
PAIRS = [(t, t) for t in TYPES] + [(torch.float32, torch.bfloat16)]
WIDTHS = [1, 2, 7, 8, 9, 31, 64, 250, 256, 257, 1000, 1001, 2047, 2048, 2056, 4096, 8192, 8200, 16384, 16392, 65536]


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(gen, *shape, dtype=torch.float32, pad=0, shift=0):
    """Normal values; pad: unused elements after each row; shift: elements before the first one."""
    rows, cols = shape
    buf = torch.full((shift + rows * (cols + pad),), 7.5, dtype=dtype, device="cuda")
    x = buf[shift:].view(rows, cols + pad)[:, :cols]
    x.copy_(torch.randn(shape, generator=gen, device="cuda"))
    return x


# --------------------------------------------------------------------------- lookup


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("H", WIDTHS)
def test_lookup(rlk, dtype, out, H):
    gen = rng(H)
    V = 37
    for T, pad, shift, scale in ((1, 0, 0, 1.0), (5, 0, 0, 8.0), (133, 8, 0, 1.0), (66, 3, 1, -0.3)):
        table = randn(gen, V, H, dtype=dtype, pad=pad, shift=shift)
        ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
        got = rlk.embedding_fwd(table, ids, scale=scale, out_dtype=out)
        assert got.dtype is out
        want, tol = ref.lookup(table, ids, scale, 0, V)
        ref.close(got, want, ref.rounded(want, out, tol))


def test_lookup_ids(rlk):
    """Padding and other shards' tokens are zero rows, others outside the vocabulary NaN rows with the flag."""
    gen = rng(1)
    V, H, n = 300, 72, 280
    table = randn(gen, V, H, dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 279, -1, 5, -1, 150], device="cuda")
    whole = rlk.embedding_fwd(table, ids, V_true=n, scale=3.0, err_flag=err)
    want, tol = ref.lookup(table, ids, 3.0, 0, n)
    ref.close(whole, want, ref.rounded(want, torch.bfloat16, tol))
    parts = [rlk.embedding_fwd(table[a:b], ids, V_true=n, vocab_start=a, scale=3.0, err_flag=err)
             for a, b in ((0, 128), (128, 256), (256, 300))]
    assert torch.equal(sum(p.float() for p in parts), whole.float())
    assert int(err) == 0
    bad = torch.tensor([0, n, -2, 299, 1 << 40, -(1 << 62), 7], device="cuda")
    got = rlk.embedding_fwd(table, bad, V_true=n, err_flag=err)
    want, tol = ref.lookup(table, bad, 1.0, 0, n)
    ref.close(got, want, ref.rounded(want, torch.bfloat16, tol))
    assert int(err) == rlk.RLK_FLAG_BAD_TARGET
    rlk.embedding_fwd(table, bad, V_true=n)                       # without a flag
    assert rlk.embedding_fwd(table, bad[:0]).shape == (0, H)


def test_lookup_special_values(rlk):
    """Infinities, NaN, overflow in the product and the smallest values go the way of fp32 and one rounding."""
    v = [0.0, -0.0, math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-45, 6e-8, 65504.0, 1.0, 2.0 ** -24]
    for dtype in TYPES:
        table = torch.tensor([v, v[::-1]], device="cuda").to(dtype)
        for scale in (1.0, 4.0, 0.25):
            got = rlk.embedding_fwd(table, torch.tensor([0, 1], device="cuda"), scale=scale)
            want = (table.float() * scale).to(dtype)
            assert torch.equal(got.view(torch.int32 if dtype is torch.float32 else torch.int16)[~want.isnan()],
                               want.view(torch.int32 if dtype is torch.float32 else torch.int16)[~want.isnan()])
            assert torch.equal(got.isnan(), want.isnan())


@pytest.mark.parametrize("H", [64, 65])
def test_lookup_layouts(rlk, H):
    """The same bits at every alignment and row distance, and nothing beside the rows is written."""
    gen = rng(3)
    V, T = 50, 40
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    for dtype, out in PAIRS:
        base = randn(rng(5), V, H, dtype=dtype)
        want = rlk.embedding_fwd(base, ids, scale=1.7, out_dtype=out)
        for shift in range(4):
            table = randn(rng(5), V, H, dtype=dtype, pad=shift, shift=shift)
            assert torch.equal(table, base)
            for oshift in (0, 1, 3, 8):
                buf = torch.full((oshift + T * (H + oshift),), 9.0, dtype=out, device="cuda")
                to = buf[oshift:].view(T, H + oshift)[:, :H]
                assert rlk.embedding_fwd(table, ids, scale=1.7, out=to) is to
                assert torch.equal(to, want)
                assert float((buf == 9.0).sum()) >= oshift * (T + 1)
                buf[oshift:].view(T, H + oshift)[:, :H] = 9.0
                assert bool((buf == 9.0).all())


def test_lookup_far_rows(rlk):
    """Rows beyond 2^31 elements."""
    V, H = (1 << 21) + 9, 1032
    table = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, (1 << 21) - 1, V - 2], device="cuda")
    table[ids] = randn(rng(1), 4, H, dtype=torch.bfloat16)
    assert torch.equal(rlk.embedding_fwd(table, ids), table[ids])


# --------------------------------------------------------------------------- the table's gradient


def many_tokens(gen, T, V, kind):
    if kind == "even":
        return torch.randint(0, V, (T,), generator=gen, device="cuda")
    if kind == "one":
        return torch.full((T,), V - 1, device="cuda")
    if kind == "runs":  # tokens that come 1, 15, 16, 17, 31, 32, 33, ... times, and the last one as often as there is room
        n = torch.tensor([1, 15, 31, 16, 32, 33, 17, 63, 64, 65, 1, 96, 97, 2, 127, 128, 129, 255, 256, 257], device="cuda")
        n = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
        x = torch.full((T,), V - 1, device="cuda")
        x[:min(T, len(n))] = n[:T] % V
        return x[torch.randperm(T, generator=gen, device="cuda")]
    x = torch.exp(torch.rand(T, generator=gen, device="cuda") * math.log(V)).long().clamp(max=V) - 1
    return torch.where(torch.rand(T, generator=gen, device="cuda") < 0.1, -1, x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,V,kind", [
    (1, 8, 1, "one"), (1, 1, 1, "one"), (2, 64, 5, "even"), (31, 7, 3, "even"), (33, 256, 1, "one"), (64, 256, 4096, "zipf"),
    (700, 40, 20, "runs"), (700, 2056, 20, "runs"), (2500, 264, 30, "runs"), (255, 72, 9, "runs"), (256, 4096, 50, "zipf"),
    (256, 30, 3000, "one"), (257, 72, 5000, "even"), (10, 16, 3000000, "even"), (1000, 257, 300, "even"), (1024, 64, 1 << 18, "zipf"),
    (1025, 64, (1 << 18) - 1, "zipf"), (3000, 4096, 151936, "zipf"), (5000, 4104, 4000, "even"), (4097, 1001, 511, "zipf"),
    (8192, 520, 512, "zipf"), (9000, 264, 50257, "one"), (20000, 16, 1000, "runs"), (16385, 24, 1 << 20, "even"),
    (300, 8200, 100, "zipf"), (300, 65536, 7, "runs"), (200000, 8, 151936, "zipf"), (100, 2, 1 << 24, "even")])
def test_table_gradient(rlk, dtype, T, H, V, kind):
    gen = rng(T + H)
    dout = randn(gen, T, H, dtype=dtype)
    ids = many_tokens(gen, T, V, kind)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = rlk.embedding_bwd(dout, ids, V, scale=0.7, err_flag=err)
    want, tol = ref.table_grad(dout, ids, V, 0.7, 0, V, None)
    ref.close(got, want, tol + ref.TINY[torch.float32], "new")
    assert int(err) == 0
    before = torch.randn((V, H), generator=gen, device="cuda") if V * H < 1 << 28 else torch.ones((V, H), device="cuda")
    added = before.clone()
    assert rlk.embedding_bwd(dout, ids, V, scale=0.7, out=added, accumulate=True) is added
    want, tol = ref.table_grad(dout, ids, V, 0.7, 0, V, before)
    ref.close(added, want, tol, "added")
    none = torch.ones(V, dtype=torch.bool, device="cuda")
    none[ids[ids >= 0]] = False
    assert torch.equal(added[none], before[none])
    assert torch.equal(got, rlk.embedding_bwd(dout, ids, V, scale=0.7))          # the same bits again


@pytest.mark.parametrize("H", [1, 3, 5, 127, 129, 255, 260, 513, 520, 640, 768, 776, 1030, 1288, 1544, 1800, 2040, 2047, 2056, 2600, 4097])
def test_table_gradient_zero_rows(rlk, H):
    """Rows without a token, at widths that leave a CTA's threads unevenly divided over them."""
    for T, V in ((3, 50), (3, 3000), (300, 70), (300, 3000)):
        ids = torch.arange(T, device="cuda") * 2 % V
        dout = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
        buf = torch.full((V * H + 16,), 7.0, device="cuda")
        got = rlk.embedding_bwd(dout, ids, V, out=buf[8:8 + V * H].view(V, H))
        assert torch.equal(got, torch.bincount(ids, minlength=V).float()[:, None].expand(V, H))
        assert bool((buf[:8] == 7.0).all()) and bool((buf[8 + V * H:] == 7.0).all())


def test_table_gradient_ids(rlk):
    """Padding and other shards add nothing, what is no token neither (flagged); shards give the rows of the whole."""
    gen = rng(4)
    T, H, V, n = 900, 136, 300, 290
    dout = randn(gen, T, H, dtype=torch.bfloat16)
    ids = many_tokens(gen, T, n, "zipf")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole = rlk.embedding_bwd(dout, ids, V, V_true=n, err_flag=err)
    for a, b in ((0, 1), (1, 128), (128, 256), (256, 300)):
        part = rlk.embedding_bwd(dout, ids, b - a, vocab_start=a, V_true=n, err_flag=err)
        assert torch.equal(part, whole[a:b])
    far = rlk.embedding_bwd(dout, ids, 64, vocab_start=V, V_true=1000, err_flag=err)   # a shard without a token
    assert not far.any()
    assert int(err) == 0
    bad = ids.clone()
    bad[::3] = torch.tensor([n, -2, 1 << 40, -(1 << 50)], device="cuda").repeat(75)
    got = rlk.embedding_bwd(dout, bad, V, V_true=n, err_flag=err)
    assert int(err) == rlk.RLK_FLAG_BAD_TARGET
    assert torch.equal(got, rlk.embedding_bwd(dout, torch.where((bad < 0) | (bad >= n), -1, bad), V, V_true=n))
    assert not rlk.embedding_bwd(dout, torch.full_like(ids, -1), V).any()
    for add in (False, True):
        w = torch.full((V, H), 3.0, device="cuda")
        rlk.embedding_bwd(dout[:0], ids[:0], V, out=w, accumulate=add)
        assert bool((w == (3.0 if add else 0.0)).all())


@pytest.mark.parametrize("H", [64, 65, 2064])
def test_table_gradient_layouts(rlk, H):
    """The same bits for every alignment and row distance; a token's row does not depend on the other tokens."""
    T, V = 333, 41
    ids = many_tokens(rng(2), T, V, "zipf")
    for dtype in TYPES:
        base = randn(rng(7), T, H, dtype=dtype)
        want = rlk.embedding_bwd(base, ids, V)
        for shift in (1, 2, 3):
            dout = randn(rng(7), T, H, dtype=dtype, pad=shift, shift=shift)
            assert torch.equal(rlk.embedding_bwd(dout, ids, V), want)
            buf = torch.full((V * H + 8,), 5.0, device="cuda")
            rlk.embedding_bwd(dout, ids, V, out=buf[shift:shift + V * H].view(V, H))
            assert torch.equal(buf[shift:shift + V * H].view(V, H), want)
            assert bool((buf[:shift] == 5.0).all()) and bool((buf[shift + V * H:] == 5.0).all())
        hot = int(torch.mode(ids[ids >= 0]).values)
        only = rlk.embedding_bwd(base[ids == hot], ids[ids == hot], V)
        assert torch.equal(only[hot], want[hot])


def test_table_gradient_far_rows(rlk):
    """dW and dout beyond 2^31 elements."""
    V, H, T = (1 << 19) + 3, 4104, (1 << 19) + 64
    dout = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T,), -1, device="cuda")
    at = torch.tensor([0, T - 1, T - 2, 5], device="cuda")
    dout[at] = randn(rng(2), 4, H, dtype=torch.bfloat16)
    ids[at] = torch.tensor([V - 1, V - 1, V - 2, 0], device="cuda")
    dW = torch.zeros((V, H), device="cuda")
    rlk.embedding_bwd(dout, ids, V, out=dW, accumulate=True)
    assert torch.equal(dW[V - 1], dout[0].float() + dout[T - 1].float())
    assert torch.equal(dW[V - 2], dout[T - 2].float()) and torch.equal(dW[0], dout[5].float())
    assert int((dW != 0).any(1).sum()) == 3


# --------------------------------------------------------------------------- layer norm


def norm_inputs(gen, T, H, dtype, out, wdtype, pad=0, shift=0):
    x = randn(gen, T, H, dtype=dtype, pad=pad, shift=shift)
    x.copy_(x.float() * (0.3 + torch.rand((T, 1), generator=gen, device="cuda")) + torch.randn((T, 1), generator=gen, device="cuda"))
    w = (1 + 0.3 * torch.randn(H, generator=gen, device="cuda")).to(wdtype)
    b = torch.randn(H, generator=gen, device="cuda").to(wdtype)
    return x, w, b, randn(gen, T, H, dtype=out, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("H", WIDTHS)
def test_norm(rlk, dtype, out, H):
    gen = rng(H)
    for T, centered, affine, wdtype, eps, pad, shift in (
            (1, True, True, dtype, 1e-5, 0, 0), (3, False, True, dtype, 1e-6, 0, 0), (130, True, True, torch.float32, 1e-5, 8, 0),
            (67, False, False, dtype, 1e-2, 3, 1), (9, True, False, dtype, 1e-5, 0, 0)):
        x, w, b, dy = norm_inputs(gen, T, H, dtype, out, wdtype, pad, shift)
        w, b = (w, b if centered else None) if affine else (None, None)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, eps=eps, centered=centered, out_dtype=out, err_flag=err)
        (wy, wm, wr), (ty, tm, tr) = ref.norm(x, w, b, eps, centered)
        assert y.dtype is out and int(err) == 0
        ref.close(y, wy, ref.rounded(wy, out, ty), "y")
        ref.close(rstd, wr, tr, "rstd")
        if centered:
            ref.close(mean, wm, tm + ref.TINY[torch.float32], "mean")
        else:
            assert mean is None
        dx, dw, db = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        want, tol = ref.norm_grad(dy, x, w, mean, rstd)
        ref.close(dx, want[0], ref.rounded(want[0], dtype, tol[0]), "dx")
        ref.close(dw, want[1], tol[1] + ref.TINY[torch.float32], "dw")
        ref.close(db, want[2], tol[2] + ref.TINY[torch.float32], "db")


@pytest.mark.parametrize("T,H", [(151, 64), (152, 64), (153, 64), (304, 256), (1300, 1001), (5000, 2048), (20000, 8), (3000, 4096)])
def test_norm_many_rows(rlk, T, H):
    for dtype, out in PAIRS:
        x, w, b, dy = norm_inputs(rng(T), T, H, dtype, out, dtype)
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, out_dtype=out)
        (wy, _, _), (ty, _, _) = ref.norm(x, w, b, 1e-5, True)
        ref.close(y, wy, ref.rounded(wy, out, ty), "y")
        got = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        want, tol = ref.norm_grad(dy, x, w, mean, rstd)
        for g, a, t, name in zip(got, want, tol, ("dx", "dw", "db")):
            ref.close(g, a, ref.rounded(a, g.dtype, t), name)
        again = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        assert all(torch.equal(g, a) for g, a in zip(got, again))
        # each of them alone, and the same
        for k, name in enumerate(("want_dx", "want_dw", "want_db")):
            one = rlk.layer_norm_bwd(dy, x, w, mean, rstd, **{n: n == name for n in ("want_dx", "want_dw", "want_db")})
            assert torch.equal(one[k], got[k]) and sum(o is not None for o in one) == 1


def test_norm_gradient_against_differences(rlk):
    """The gradients of a sum of y times a constant, from the forward alone: fp32 forwards of about 2^-24 and
    steps of 2^-7 leave 2^-16 of noise a value and 2^-14 of curvature."""
    T, H = 3, 24
    gen = rng(8)
    x, w, b, dy = norm_inputs(gen, T, H, torch.float32, torch.float32, torch.float32)
    for centered in (True, False):
        bias = b if centered else None

        def loss(x, w, bias):
            y, _, _ = rlk.layer_norm_fwd(x, w, bias, centered=centered)
            return float((y.double() * dy.double()).sum())

        _, mean, rstd = rlk.layer_norm_fwd(x, w, bias, centered=centered)
        dx, dw, db = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        step = 2.0 ** -7
        for k, (t, g) in enumerate(((x, dx), (w, dw), (bias, db))):
            if t is None:
                continue
            for i in range(0, t.numel(), 5):
                e = torch.zeros(t.numel(), device="cuda")
                e[i] = step
                up, down = [x, w, bias], [x, w, bias]
                up[k], down[k] = t + e.view(t.shape), t - e.view(t.shape)
                diff = (loss(*up) - loss(*down)) / (2 * step)
                assert abs(diff - float(g.flatten()[i])) < 2e-3 * (1 + abs(diff)), (centered, k, i)


@pytest.mark.parametrize("H", [64, 65, 2048, 8200])
def test_norm_layouts(rlk, H):
    """The same bits at every alignment and row distance, in place and in any batch; nothing beside the rows is written."""
    T = 21
    for dtype, out in PAIRS:
        x, w, b, dy = norm_inputs(rng(3), T, H, dtype, out, dtype)
        y, mean, rstd = rlk.layer_norm_fwd(x, w, b, out_dtype=out)
        grads = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
        for shift in (1, 3, 8):
            x2, w2, b2, dy2 = norm_inputs(rng(3), T, H, dtype, out, dtype, pad=shift, shift=shift)
            x2, dy2 = x2.copy_(x), dy2.copy_(dy)
            w2 = torch.cat([w[:1], w])[1:]
            buf = torch.full((shift + T * (H + shift),), 9.0, dtype=out, device="cuda")
            to = buf[shift:].view(T, H + shift)[:, :H]
            y2, mean2, rstd2 = rlk.layer_norm_fwd(x2, w2, b, out=to)
            assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
            to.fill_(9.0)
            assert bool((buf == 9.0).all())
            buf = torch.full((shift + T * (H + shift),), 9.0, dtype=dtype, device="cuda")
            to = buf[shift:].view(T, H + shift)[:, :H]
            got = rlk.layer_norm_bwd(dy2, x2, w2, mean, rstd, out=to)
            assert all(torch.equal(a, g) for a, g in zip(got, grads))
            to.fill_(9.0)
            assert bool((buf == 9.0).all())
        odd = torch.empty(T * H + 1, dtype=dtype, device="cuda")[1:].view(T, H).copy_(x)
        for centered in (True, False):                       # without weights
            bare = [rlk.layer_norm_fwd(v, centered=centered, out_dtype=out) for v in (x, odd)]
            assert torch.equal(bare[0][0], bare[1][0]) and torch.equal(bare[0][2], bare[1][2])
            bare = [rlk.layer_norm_bwd(dy, v, None, bare[0][1], bare[0][2]) for v in (x, odd)]
            assert all(torch.equal(p, q) for p, q in zip(*bare))
        some = rlk.layer_norm_fwd(x[5:9], w, b, out_dtype=out)
        assert torch.equal(some[0], y[5:9]) and torch.equal(some[1], mean[5:9])
        assert torch.equal(rlk.layer_norm_bwd(dy[5:9], x[5:9], w, mean[5:9], rstd[5:9])[0], grads[0][5:9])
        if dtype is out:
            z = x.clone()
            assert rlk.layer_norm_fwd(z, w, b, out=z)[0] is z and torch.equal(z, y)
            z = dy.clone()
            assert torch.equal(rlk.layer_norm_bwd(z, x, w, mean, rstd, out=z)[0], grads[0])
        z = x.clone()
        assert torch.equal(rlk.layer_norm_bwd(dy, z, w, mean, rstd, out=z)[0], grads[0])


def test_norm_side_by_side(rlk):
    """Column slices of one buffer, as a result and its input."""
    x, w, b, _ = norm_inputs(rng(3), 12, 64, torch.float32, torch.float32, torch.float32)
    buf = torch.zeros((12, 200), device="cuda")
    buf[:, :64] = x
    y, _, _ = rlk.layer_norm_fwd(buf[:, :64], w, b, out=buf[:, 64:128])
    assert torch.equal(y, rlk.layer_norm_fwd(x, w, b)[0]) and torch.equal(buf[:, :64], x) and not buf[:, 128:].any()
    with pytest.raises(rlk.RlkError):
        rlk.layer_norm_fwd(buf[:, :64], w, b, out=buf[:, 63:127])


@pytest.mark.parametrize("H", [8, 100, 4096, 16384, 20000])
def test_norm_far_values(rlk, H):
    """Offsets much larger than what varies, and rows whose sums and squares are beyond fp32."""
    gen = rng(H)
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.randn((6, H), generator=gen, device="cuda")
        rows = [z[0] + 1000.0, z[1] * 1e30, z[2] * 1e36, z[3] * 1e-30, torch.full_like(z[4], 3e38), z[5] * 1e-3 - 64.0]
        x = torch.stack(rows).to(dtype)
        for centered in (True, False):
            y, mean, rstd = rlk.layer_norm_fwd(x, centered=centered)
            (wy, wm, wr), (ty, tm, tr) = ref.norm(x, None, None, 1e-5, centered)
            # rstd of the rows beyond 2^126 is below fp32's normal values: half of the smallest one
            ref.close(rstd, wr, tr + ref.TINY[torch.float32], "rstd")
            ref.close(y, wy, ref.rounded(wy, dtype, ty), "y")
            if centered:
                ref.close(mean, wm, tm, "mean")


def test_norm_rows_of_nothing(rlk):
    """Rows of zeros and of one value, and rows with NaN or infinities: NaN throughout, flagged, and no other row."""
    for H in (5, 64, 9000):
        x = torch.randn((6, H), generator=rng(1), device="cuda")
        x[1] = 0.0
        x[2] = 4.25
        y, mean, rstd = rlk.layer_norm_fwd(x)
        (wy, _, wr), (ty, _, tr) = ref.norm(x, None, None, 1e-5, True)
        ref.close(y, wy, ty + 2e-7, "y")
        ref.close(rstd, wr, tr, "rstd")
        for bad in (math.nan, math.inf, -math.inf):
            for centered in (True, False):
                z = x.clone()
                z[3, H // 2] = bad
                err = torch.zeros(1, dtype=torch.int32, device="cuda")
                good, gm, gr = rlk.layer_norm_fwd(x, centered=centered, err_flag=err)
                assert int(err) == 0
                y, mean, rstd = rlk.layer_norm_fwd(z, centered=centered, err_flag=err)
                assert int(err) == rlk.RLK_FLAG_NONFINITE
                assert bool(y[3].isnan().all()) and bool(rstd[3].isnan())
                keep = torch.arange(6, device="cuda") != 3
                assert torch.equal(y[keep], good[keep]) and torch.equal(rstd[keep], gr[keep])
                dx, _, _ = rlk.layer_norm_bwd(x, z, None, mean, rstd)
                assert bool(dx[3].isnan().all()) and bool(dx[keep].isfinite().all())


def test_norm_empty_batch(rlk):
    x = torch.randn((0, 40), device="cuda")
    w = torch.ones(40, device="cuda")
    y, mean, rstd = rlk.layer_norm_fwd(x, w)
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    dx, dw, db = rlk.layer_norm_bwd(x, x, w, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any() and dw.shape == (40,)


def test_norm_far_rows(rlk):
    """Rows beyond 2^31 elements (a row distance of 2^27)."""
    T, H, ld = 20, 256, 1 << 27
    buf = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, H), (ld, 1))
    x.copy_(torch.randn((T, H), generator=rng(1), device="cuda"))
    y, mean, rstd = rlk.layer_norm_fwd(x)
    near = x.contiguous()
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd), rlk.layer_norm_fwd(near)))
    want = rlk.layer_norm_bwd(y, near, None, mean, rstd)
    got = rlk.layer_norm_bwd(y, x, None, mean, rstd, out=x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# --------------------------------------------------------------------------- all gradients


def gradients(gen, sizes, dtype, shift=0):
    n = sum(sizes)
    flat = torch.randn(n + shift, generator=gen, device="cuda").to(dtype)
    return list(flat[shift:].split(sizes)), flat


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("sizes", [[1], [7], [8], [0], [0, 5, 0], [4095, 1, 4097], [8191, 8192, 8193], [100000], [3, 5] * 20,
                                   [1000] * 33, [17] * 700, [0] * 600 + [300], [2500000, 11, 4100001]])
def test_clip(rlk, dtype, out, sizes):
    grads, flat = gradients(rng(len(sizes)), sizes, dtype)
    want, rel = ref.total_norm(grads)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    norm = rlk.grad_norm(grads, err_flag=err)
    assert norm.shape == () and abs(float(norm) - want) <= rel * want
    for max_norm in (0.3 * want + 1e-9, 3 * want + 1, math.inf):
        outs = [torch.empty_like(g, dtype=out) for g in grads]
        got = rlk.clip_grad_norm(grads, max_norm, out=outs, err_flag=err)
        assert torch.equal(got, norm)
        f = min(1.0, max_norm / want) if want else 1.0
        for g, o in zip(grads, outs):
            exact = g.double() * f
            ref.close(o, exact, ref.rounded(exact, out, exact.abs() * (rel + 2 * ref.U) if f < 1 else 0 * exact))
        if dtype is out:
            mine = [g.clone() for g in grads]
            assert torch.equal(rlk.clip_grad_norm(mine, max_norm), norm)
            assert all(torch.equal(a, b) for a, b in zip(mine, outs))
    assert int(err) == 0


def test_clip_mixed_types(rlk):
    """Types, shapes, alignments and both kinds of results in one call; the norm's bits at every alignment."""
    gen = rng(5)
    grads, to = [], []
    for i, (shape, dtype, out) in enumerate([((3, 5), torch.float32, torch.float32), ((4100,), torch.bfloat16, torch.bfloat16),
                                            ((2, 3, 1111), torch.float16, torch.float16), ((90000,), torch.float32, torch.bfloat16),
                                            ((), torch.float32, torch.float32), ((257, 33), torch.bfloat16, torch.bfloat16)] * 7):
        grads.append(torch.randn(shape, generator=gen, device="cuda").to(dtype))
        to.append(torch.empty(shape, dtype=out, device="cuda") if i % 3 else (grads[-1] if dtype is out else torch.empty(shape, dtype=out, device="cuda")))
    want, rel = ref.total_norm(grads)
    norm = rlk.grad_norm(grads)
    assert abs(float(norm) - want) <= rel * want
    for shift in range(1, 8):
        moved = [torch.empty(g.numel() + shift, dtype=g.dtype, device="cuda")[shift:].view(g.shape).copy_(g) for g in grads]
        assert torch.equal(rlk.grad_norm(moved), norm)
    before = [g.clone() for g in grads]
    assert torch.equal(rlk.clip_grad_norm(grads, want / 3, out=to), norm)
    for g, o in zip(before, to):
        exact = g.double() / 3
        ref.close(o, exact, ref.rounded(exact, o.dtype, exact.abs() * (rel + 2 * ref.U)))
    assert abs(float(rlk.grad_norm(grads[:1] + grads[:1])) - math.sqrt(2) * float(grads[0].double().norm())) < 1e-5
    assert torch.equal(rlk.grad_norm(grads[1]), rlk.grad_norm([grads[1]]))


def test_clip_values(rlk):
    """Squares beyond fp32 on both sides, and norms that are not finite: nothing is scaled, and the flag says so."""
    gen = rng(6)
    z = torch.randn(5000, generator=gen, device="cuda")
    for f in (1e-38, 1e-30, 1e-20, 1e-15, 1e15, 1e20, 1e30, 1e36):
        for dtype in (torch.float32, torch.bfloat16):
            grads = [(z * f).to(dtype), (z[:33] * f * 1e-3).to(dtype)]
            want, rel = ref.total_norm(grads)
            got = rlk.grad_norm(grads)
            assert abs(float(got) - want) <= rel * want + 2.0 ** -150, f
            mixed = [(z * 1e-25).to(dtype), (z[:100] * f).to(dtype), z[:1] * 0]
            want, rel = ref.total_norm(mixed)
            assert abs(float(rlk.grad_norm(mixed)) - want) <= rel * want + 2.0 ** -150, f
    for bad in (math.nan, math.inf, -math.inf, 3e38):
        g = z.clone()
        g[4321] = bad
        if bad == 3e38:
            g[:4000] = bad                     # finite gradients, a norm beyond fp32
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mine, out = g.clone(), torch.empty_like(g)
        norm = rlk.clip_grad_norm(mine, 1.0, err_flag=err)
        assert not bool(norm.isfinite()) and int(err) == rlk.RLK_FLAG_NONFINITE
        rlk.clip_grad_norm(g, 1.0, out=out)
        for x in (mine, out):
            assert torch.equal(x.view(torch.int32), g.view(torch.int32))
        err.zero_()
        assert not bool(rlk.grad_norm(g, err_flag=err).isfinite()) and int(err) == rlk.RLK_FLAG_NONFINITE
    zero = torch.zeros(100, device="cuda")
    assert float(rlk.clip_grad_norm(zero, 1.0)) == 0.0 and not zero.any()


def test_norm_of_many_elements(rlk):
    """2^32 equal elements, 535 chunks a thread. Relative to the sum of squares: 17 roundings of a chunk's, 2 of the sum of chunks,
    whose losses are kept, 8 in a warp and between warps, as many where the shares are joined (3 sums with their losses, 8)
    and the root's: 38 half steps at most, of which the root leaves 19."""
    g = torch.full((1 << 32,), 0.0123, dtype=torch.bfloat16, device="cuda")
    want = 65536 * float(g[0])
    assert abs(float(rlk.grad_norm([g])) / want - 1) <= 20 * ref.U


def test_clip_far_elements(rlk):
    """A tensor of more than 2^31 elements."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    g[at] = torch.tensor([1.0, 2.0, 4.0, 2.0], device="cuda").bfloat16()
    assert float(rlk.clip_grad_norm(g, 2.5)) == 5.0
    assert g[at].tolist() == [0.5, 1.0, 2.0, 1.0] and float(g.float().abs().sum()) == 4.5


# --------------------------------------------------------------------------- calls


def test_refusals(rlk):
    """What the binding refuses before anything runs."""
    x = torch.ones((4, 16), device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.ones(16, device="cuda")
    r = torch.ones(4, device="cuda")
    for e, f in (
            (ValueError, lambda: rlk.embedding_fwd(x.cpu(), ids)), (ValueError, lambda: rlk.embedding_fwd(x, ids.cpu())),
            (TypeError, lambda: rlk.embedding_fwd(x, ids.int())), (ValueError, lambda: rlk.embedding_fwd(x, ids[:, None])),
            (TypeError, lambda: rlk.embedding_fwd(x.double(), ids)), (ValueError, lambda: rlk.embedding_fwd(x.t(), ids)),
            (ValueError, lambda: rlk.embedding_fwd(x, ids, out=x[:, :8])), (rlk.RlkError, lambda: rlk.embedding_fwd(x, ids, out=x)),
            (rlk.RlkError, lambda: rlk.embedding_fwd(x, ids, V_true=0)), (rlk.RlkError, lambda: rlk.embedding_fwd(x, ids, vocab_start=-1)),
            (rlk.RlkError, lambda: rlk.embedding_fwd(x, ids, scale=math.nan)), (rlk.RlkError, lambda: rlk.embedding_fwd(x.half(), ids, out_dtype=torch.float32)),
            (ValueError, lambda: rlk.embedding_bwd(x, ids[:3], 4)), (ValueError, lambda: rlk.embedding_bwd(x, ids, 4, accumulate=True)),
            (ValueError, lambda: rlk.embedding_bwd(x, ids, 4, out=torch.ones((5, 16), device="cuda"))),
            (TypeError, lambda: rlk.embedding_bwd(x, ids, 4, out=x.half())), (rlk.RlkError, lambda: rlk.embedding_bwd(x, ids, 4, out=x)),
            (ValueError, lambda: rlk.embedding_bwd(x.repeat(100, 1), ids.repeat(100), 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
            (rlk.RlkError, lambda: rlk.embedding_bwd(x, ids, 0)),
            (TypeError, lambda: rlk.layer_norm_fwd(x, w.half())), (TypeError, lambda: rlk.layer_norm_fwd(x.half(), w, w.half())),
            (ValueError, lambda: rlk.layer_norm_fwd(x, w[:8])), (rlk.RlkError, lambda: rlk.layer_norm_fwd(x, w, eps=0.0)),
            (ValueError, lambda: rlk.layer_norm_fwd(x[0], w)), (rlk.RlkError, lambda: rlk.layer_norm_fwd(x, w, out_dtype=torch.float16)),
            (ValueError, lambda: rlk.layer_norm_bwd(x[:3], x, w, r, r)), (ValueError, lambda: rlk.layer_norm_bwd(x, x, w, r, r[:3])),
            (ValueError, lambda: rlk.layer_norm_bwd(x, x, w, r, r, want_dx=False, want_dw=False, want_db=False)),
            (ValueError, lambda: rlk.layer_norm_bwd(x, x, w, r, r, want_dx=False, out=x.clone())),
            (TypeError, lambda: rlk.layer_norm_bwd(x, x, w, r, r, out=x.half())),
            (ValueError, lambda: rlk.grad_norm([])), (ValueError, lambda: rlk.grad_norm([x, x.cpu()])),
            (ValueError, lambda: rlk.grad_norm([x.t()])), (TypeError, lambda: rlk.grad_norm([x.double()])),
            (TypeError, lambda: rlk.grad_norm([x, None])), (ValueError, lambda: rlk.clip_grad_norm([x], 0.0)),
            (ValueError, lambda: rlk.clip_grad_norm([x], math.nan)), (ValueError, lambda: rlk.clip_grad_norm([x], 1.0, out=[])),
            (ValueError, lambda: rlk.clip_grad_norm([x], 1.0, out=[x[:2]])), (rlk.RlkError, lambda: rlk.clip_grad_norm([x, x], 1.0)),
            (rlk.RlkError, lambda: rlk.clip_grad_norm([x.half()], 1.0, out=[torch.empty_like(x)])),
            (rlk.RlkError, lambda: rlk.clip_grad_norm([x[:2], x[2:]], 1.0, out=[x[1:3], x[2:]]))):
        with pytest.raises(e):
            f()


def all_calls(rlk, d, stream=None):
    """Every entry point once."""
    k = dict(stream=stream)
    o = [rlk.embedding_fwd(d["table"], d["ids"], scale=2.0, **k), rlk.embedding_bwd(d["dy"], d["ids"], d["table"].shape[0], **k)]
    y, mean, rstd = rlk.layer_norm_fwd(d["x"], d["w"], d["b"], **k)
    o += [y, mean, rstd, *rlk.layer_norm_bwd(d["dy"], d["x"], d["w"], mean, rstd, **k)]
    o.append(rlk.grad_norm([d["x"], d["dy"], d["w"]], **k))
    out = [torch.empty_like(g) for g in (d["x"], d["dy"])]
    o += [rlk.clip_grad_norm([d["x"], d["dy"]], 1.0, out=out, **k), *out]
    return o


def call_inputs(T=600, H=520, V=90, seed=0):
    gen = rng(seed)
    x, w, b, dy = norm_inputs(gen, T, H, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    return dict(table=randn(gen, V, H, dtype=torch.bfloat16), ids=many_tokens(gen, T, V, "zipf"), x=x, w=w, b=b, dy=dy)


def test_other_stream(rlk):
    d = call_inputs()
    want = all_calls(rlk, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = all_calls(rlk, d, s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two calls at once, each with a workspace of its own
    t = torch.cuda.Stream()
    other = call_inputs(seed=1)
    want2 = all_calls(rlk, other)
    torch.cuda.synchronize()
    got, got2 = all_calls(rlk, d, s), all_calls(rlk, other, t)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(got2, want2))


def test_graphs_sharing_a_pool(rlk):
    """Captured, replayed with new inputs, and two graphs of one pool in turn."""
    d, other = call_inputs(), call_inputs(seed=1)
    want, want2 = all_calls(rlk, d), all_calls(rlk, other)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        got = all_calls(rlk, d)
    kept = [g.clone() for g in want]
    with torch.cuda.graph(two, pool=one.pool()):
        got2 = all_calls(rlk, other)
    for _ in range(3):
        one.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        two.replay()
        assert all(torch.equal(a, b) for a, b in zip(got2, want2))
    for k in d:
        d[k].copy_(other[k])
    one.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want2))
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_dirty_workspaces(rlk):
    """What a workspace holds before a call does not matter, nor that it is larger than it must be."""
    d = call_inputs()
    T, H = d["x"].shape
    _, mean, rstd = rlk.layer_norm_fwd(d["x"], d["w"], d["b"])
    ids = torch.full_like(d["ids"], 3)
    for fill in (0, 255, 127):
        for f in (lambda **k: rlk.embedding_bwd(d["dy"], ids, 90, **k), lambda **k: rlk.grad_norm([d["x"]], **k),
                  lambda **k: rlk.layer_norm_bwd(d["dy"], d["x"], d["w"], mean, rstd, **k)):
            n = max(rlk.embedding_bwd_workspace_bytes(T, H), rlk.layer_norm_bwd_workspace_bytes(T, H), rlk.grad_norm_workspace_bytes(1)) + 77
            ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
            got, want = f(workspace=ws), f()
            for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
                assert torch.equal(a, b)


def test_autograd(rlk):
    """The differentiable forms against torch's own in fp64."""
    gen = rng(9)
    T, H, V = 70, 48, 30
    table = torch.randn((V, H), generator=gen, device="cuda").requires_grad_()
    ids = many_tokens(gen, T, V, "zipf")
    w, b = (torch.randn(H, generator=gen, device="cuda").requires_grad_() for _ in range(2))
    c = torch.randn((T, H), generator=gen, device="cuda")
    for centered in (True, False):
        for t in (table, w, b):
            t.grad = None
        x = rlk.embedding(table, ids, scale=3.0)
        y = rlk.layer_norm(x, w, b, centered=centered)
        (y * c).sum().backward()
        p = [t.detach().double().requires_grad_() for t in (table, w, b)]
        x = torch.where((ids < 0)[:, None], 0.0, p[0][ids.clamp(min=0)] * 3.0)
        d = x - x.mean(1, keepdim=True) if centered else x
        y = d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * p[1] + p[2]
        (y * c.double()).sum().backward()
        for t, q in zip((table, w, b), p):
            # rows of padding have d = 0 and rstd = 316, so nothing cancels; 32 roundings of the largest terms
            assert float((t.grad.double() - q.grad).abs().max()) <= 64 * ref.U * float(q.grad.abs().max()) * math.sqrt(T)
    # an expanded gradient, a type of its own, and a second derivative
    rlk.layer_norm(rlk.embedding(table, ids), out_dtype=torch.bfloat16).sum().backward()
    half = table.detach().bfloat16().requires_grad_()
    rlk.embedding(half, ids).float().square().sum().backward()
    assert half.grad.dtype is torch.bfloat16
    x = torch.randn((4, 16), device="cuda", requires_grad=True)
    for f in (lambda: rlk.layer_norm(x), lambda: rlk.embedding(x, torch.tensor([1, 2], device="cuda")).square()):
        (d,) = torch.autograd.grad(f().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            d.square().sum().backward()


def test_autograd_sees_what_is_written(rlk):
    """In-place clipping and results written into given tensors make a backward that needs the old values fail."""
    x = torch.randn((4, 16), device="cuda")
    ids = torch.tensor([0, 1, 2, 3], device="cuda")
    for write in (lambda t: rlk.clip_grad_norm([t], 0.1), lambda t: rlk.embedding_fwd(x, ids, out=t),
                  lambda t: rlk.layer_norm_fwd(x, out=t), lambda t: rlk.embedding_bwd(x, ids, 4, out=t, accumulate=True)):
        p = torch.randn((4, 16), device="cuda", requires_grad=True)
        saved = torch.randn((4, 16), device="cuda")
        loss = (p * saved).sum()
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_step_of_a_tied_model(rlk):
    """The operators together, around linear_logp: tokens -> embedding -> norm -> head -> loss, and back into one
    weight's gradient, clipped. bf16 rounds x, h, dH and dx once each, and z's gradient dz: relative L2 below 1e-2."""
    T, H, V, n = 300, 256, 3000, 2900
    gen = rng(11)
    W = (0.1 * torch.randn((V, H), generator=gen, device="cuda")).bfloat16()
    w = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda"))
    ids = many_tokens(gen, T, n, "zipf")
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    g = torch.rand(T, generator=gen, device="cuda") / T
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = math.sqrt(H)

    x = rlk.embedding_fwd(W, ids, scale=scale, V_true=n, err_flag=err)
    h, _, rstd = rlk.layer_norm_fwd(x, w, centered=False, err_flag=err)
    logp, lse = rlk.linear_logp_fwd(h, W, y, n, err_flag=err)
    dH, dW = rlk.linear_logp_bwd(h, W, y, lse, g, n, err_flag=err)
    dx, dw, _ = rlk.layer_norm_bwd(dH, x, w, None, rstd, want_db=False, err_flag=err)
    rlk.embedding_bwd(dx, ids, V, scale=scale, V_true=n, out=dW, accumulate=True, err_flag=err)
    before = [dW.clone(), dw.clone()]
    norm = rlk.clip_grad_norm([dW, dw], 0.01, err_flag=err)
    assert int(err) == 0

    W64, w64 = W.double().requires_grad_(), w.double().requires_grad_()
    x64 = torch.where((ids < 0)[:, None], 0.0, W64[ids.clamp(min=0)] * scale)
    h64 = x64 * (x64.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w64
    want = (h64 @ W64[:n].t()).log_softmax(1).gather(1, y[:, None])[:, 0]
    (want * g.double()).sum().backward()
    assert float((logp - want.detach()).abs().max()) < 5e-2      # h in bf16: 2^-9 of |z| up to 10
    for got, exact in zip(before, (W64.grad, w64.grad)):
        assert float((got.double() - exact).norm() / exact.norm()) < 1e-2
    total = math.sqrt(float(W64.grad.square().sum() + w64.grad.square().sum()))
    assert abs(float(norm) / total - 1) < 1e-2 and total > 0.01
    for got, was in zip((dW, dw), before):
        assert float((got.double() - was.double() * (0.01 / float(norm))).abs().max()) <= 3 * ref.U * float(was.abs().max())


def test_norm_beside_the_gradients(rlk):
    """A norm in the gradients' own buffer: refused where clipping would write it under a reader."""
    g = torch.ones(101, device="cuda")
    with pytest.raises(rlk.RlkError):
        rlk.clip_grad_norm([g], 1.0, norm=g[40])
    with pytest.raises(rlk.RlkError):
        rlk.clip_grad_norm([g[:100]], 1.0, out=[g[1:]], norm=torch.empty((), device="cuda"))
    assert g.tolist() == [1.0] * 101
    rlk.clip_grad_norm([g[:100]], 5.0, norm=g[100])
    assert g.tolist() == [0.5] * 100 + [10.0]


def test_two_threads(rlk):
    """Calls from two host threads at once, on streams of their own."""
    import threading
    d = [call_inputs(seed=i) for i in range(2)]
    want = [all_calls(rlk, x) for x in d]
    torch.cuda.synchronize()
    same = [0, 0]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got = all_calls(rlk, d[i], s)
            s.synchronize()
            same[i] += all(torch.equal(a, b) for a, b in zip(got, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert same == [20, 20]


def test_captured_autograd_step(rlk):
    """Forward and backward of the differentiable forms in a graph, replayed on new tokens. No eager graph of the same
    leaves is alive when the capture starts."""
    gen = rng(12)
    T, H, V = 300, 64, 50
    table = torch.randn((V, H), generator=gen, device="cuda").requires_grad_()
    w = torch.randn(H, generator=gen, device="cuda").requires_grad_()
    ids, other = many_tokens(gen, T, V, "zipf"), many_tokens(gen, T, V, "even")

    def step():
        y = rlk.layer_norm(rlk.embedding(table, ids, scale=2.0), w, centered=False)
        return torch.autograd.grad(y.square().sum(), (table, w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for new in (ids.clone(), other):
        ids.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("T", [1024, 1025])
def test_norm_many_wide_misaligned_rows(rlk, dtype, out, T):
    """The bits of aligned rows, and those of few rows, whichever kernel takes them."""
    H = 9000
    gen = rng(13)
    x = randn(gen, T, H, dtype=dtype)
    w, b = (torch.randn(H, generator=gen, device="cuda") for _ in range(2))
    x[7] = 3e38 if dtype is not torch.float16 else 60000.0   # the sums are taken once more, at a smaller scale
    x[7, ::2] *= -1
    away = torch.empty(T * H + 1, dtype=dtype, device="cuda")[1:].view(T, H)
    away.copy_(x)
    for centered in (True, False):
        want = rlk.layer_norm_fwd(x, w, b, centered=centered, out_dtype=out)
        got = rlk.layer_norm_fwd(away, w, b, centered=centered, out_dtype=out)
        few = rlk.layer_norm_fwd(away[:9], w, b, centered=centered, out_dtype=out)
        for a, c, d in zip(want, got, few):
            assert a is None or (torch.equal(a, c) and torch.equal(a[:9], d))
