"""Rows whose logits lie far from zero -- offsets, low temperatures, masks by a finite value, s z
beyond the range of fp32 -- against plain 64-bit forms about the row's maximum M:

  d = s (z - M),  L = log sum e^d,  log p = d - L

Error of a log probability: L is off by the row sum's relative error EPS_SUM (logits_ref) and its own
rounding, d by the roundings of s, of z - M and of the product, each 2^-24 |d|; none grows with |s M|.
Where M and z are far apart, z - M or log p may leave fp32's range: then both are -inf."""
import math

import pytest
import torch

import logits_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = math.inf
TEMPERATURES = [1.0, 0.7, 0.01, 1e-3, 1e-6, 3.0]


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def far_rows(dtype, n, seed):
    """Rows far from zero; row 12 is ordinary, row 13 empty."""
    lowest = torch.finfo(dtype).min
    mask = -6e4 if dtype == torch.float16 else -1e9
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn():
        return torch.randn(n, generator=gen, device="cuda")

    hide = torch.rand((3, n), generator=gen, device="cuda") < 0.95
    col = torch.arange(n, device="cuda")
    rows = [
        torch.full((n,), lowest, device="cuda"),                     # masked wholly, by the type's lowest value
        torch.full((n,), mask, device="cuda"),                       # and by a usual one
        torch.full((n,), -3000.0, device="cuda"),
        torch.where(hide[0], lowest, randn() * 3),                   # masked partly
        torch.where(hide[1], mask, randn() * 3),
        randn() + 1000,                                              # an offset
        randn() * 2 + 30,                                            # usual logits (far at a low temperature)
        randn() * 500 - 20000,
        torch.where(col % 2 == 0, -INF, lowest),                     # masked both ways
        torch.where(col == n // 2, lowest, -INF),                    # one finite column, the lowest
        torch.full((n,), -lowest, device="cuda"),                    # the largest value everywhere
        torch.where(col % 3 == 0, 512.0, 511.0),
        randn() * 3,
        torch.full((n,), -INF, device="cuda"),
    ]
    return torch.stack(rows).to(dtype), gen


def exact(z, s):
    """(d, L, log p) in 64 bits; an empty row has log p -inf and L 0."""
    z = z.double()
    M = z.max(1, keepdim=True).values
    d = torch.where(z == -INF, z, s * (z - torch.where(M == -INF, torch.zeros_like(M), M)))
    L = torch.where(M == -INF, torch.zeros_like(M), d.exp().sum(1, keepdim=True).log())
    return d, L, d - L


def logp_tolerance(d, L):
    """Of log probabilities with this distance d from the row's maximum."""
    d = torch.where(d.isfinite(), d.abs(), torch.zeros_like(d))
    return ref.EPS_SUM + ref.EPS * (2 * d + 2 * L.abs() + 1)


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,copies", [(1, 1), (40, 1), (5003, 1), (5003, 100), (40000, 1), (40000, 30)])
def test_scores_far_from_zero(rlk, dtype, temperature, n, copies):
    z, gen = far_rows(dtype, n, seed=n)
    z = z.repeat(copies, 1)                        # other launch shapes
    T, s = z.shape[0], 1.0 / temperature
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    d, L, lp = exact(z, s)
    for k in (0, 20):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = rlk.token_logprobs(z, y, top_k=k, temperature=temperature, err_flag=err)
        at = y[:, None]
        ref.assert_within(r.logp, lp.gather(1, at)[:, 0], logp_tolerance(d.gather(1, at), L)[:, 0], "logp")
        assert not (r.logp > 0).any()
        want = ref.scores(z, n, s, y, k)           # its lse, entropy and whole numbers are safe
        lse0 = torch.where(want["lse"].isfinite(), want["lse"].abs(), torch.zeros_like(want["lse"]))
        lse = torch.where((z == -INF).all(1), want["lse"], want["lse"].clamp(min=torch.finfo(torch.float32).min))
        ref.assert_within(r.lse, lse, ref.EPS_SUM + 2 * ref.EPS * lse0, "lse")   # -inf: an empty row alone
        ref.assert_within(r.entropy, want["entropy"], ref.EPS_SUM * (2 + 2 * want["entropy"]), "entropy")
        assert torch.equal(r.rank, want["rank"])
        if k:
            assert torch.equal(r.top_ids, want["top_ids"])
            none = r.top_ids < 0
            at = r.top_ids.clamp(min=0)
            ref.assert_within(r.top_logp, lp.gather(1, at).masked_fill(none, -INF),
                              logp_tolerance(d.gather(1, at), L), "top_logp")
            assert not (r.top_logp > 0).any()
        assert int(err) == 0


def near_teacher(z, K, gen):
    """Entries among the row's best columns (a mask's log probability may leave fp32's range), some
    absent; for z of one column or more."""
    T, n = z.shape
    best = z.float().topk(min(n, 2 * K), 1).indices
    ids = best.gather(1, torch.randint(0, best.shape[1], (T, K), generator=gen, device="cuda"))
    ids = torch.where(z.gather(1, ids) < z.float().max(1, keepdim=True).values - 1e4, torch.full_like(ids, -1), ids)
    ids[::3, -1] = -1
    return ids, torch.randn((T, K), generator=gen, device="cuda") * 4 - 2000


def loss_and_tolerance(z, s, ids, t):
    d, L, lp = exact(z, s)
    q, logq, _ = ref.teacher(ids, t, z.shape[1], s)
    at = ids.clamp(min=0)
    term = logq - lp.gather(1, at)
    loss = torch.where(q > 0, q * term, torch.zeros_like(q)).sum(1)
    # q and log q: ex2, the sum over K and its logarithm (16 eps), |log q| in the exponent; then the sums
    tol = q * (logp_tolerance(d.gather(1, at), L) + ref.EPS * (16 + 4 * logq.abs()) * (1 + term.abs()))
    return loss, torch.where(q > 0, tol, torch.zeros_like(q)).sum(1) + ref.EPS


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,copies", [(1, 1), (40, 1), (5003, 1), (5003, 100), (40000, 1), (40000, 60)])
def test_distillation_loss_far_from_zero(rlk, dtype, temperature, n, copies):
    z, gen = far_rows(dtype, n, seed=n + 1)
    z = z.repeat(copies, 1)
    ids, t = near_teacher(z, 12, gen)
    s = 1.0 / temperature
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = rlk.distill_topk_fwd(z, ids, t, temperature=temperature, err_flag=err)
    want, tol = loss_and_tolerance(z, s, ids, t)
    ref.assert_within(loss, want, tol, "loss")
    g = torch.zeros(z.shape[0], device="cuda")
    loss2, lse2, _ = rlk.distill_topk_fwd_bwd(z, ids, t, g, temperature=temperature, err_flag=err)
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse)
    assert int(err) == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_mask_that_leaves_nothing_gives_a_uniform_row(rlk, dtype):
    """The divergence from one teacher token to n equal ones is log n, and no log probability is above 0."""
    n = 50257
    for value in (torch.finfo(dtype).min, -6e4, -1e4):
        z = torch.full((2, n), value, dtype=dtype, device="cuda")
        y = torch.tensor([0, n - 1], device="cuda")
        for tau in (1.0, 0.5):
            r = rlk.token_logprobs(z, y, top_k=3, temperature=tau)
            loss, _ = rlk.distill_topk_fwd(z, y[:, None], torch.zeros((2, 1), device="cuda"), temperature=tau)
            tol = ref.EPS_SUM + 2 * ref.EPS * math.log(n)
            for got, sign in ((r.logp, -1), (r.top_logp, -1), (r.entropy, 1), (loss, 1)):
                assert float((got - sign * math.log(n)).abs().max()) <= tol, (value, tau)


OUTS = [(torch.bfloat16, None), (torch.float16, None), (torch.float32, None), (torch.float32, torch.bfloat16)]


NEAR = {torch.float32: 256, torch.float16: 512, torch.bfloat16: 4096}


def p_error(d, L, lp, z, s, out):
    """(p, relative error of the kernels' p): as of a log probability, then its product with log2 e and
    ex2. Rows whose |lse| is at most NEAR may take p from the fp32 lse, which is off by 2^-24 |lse|, with
    s z rounded like it: half of that limit's 2^-23, an eighth of what the output's rounding adds in f16 and
    bf16."""
    M = z.double().max(1, keepdim=True).values.nan_to_num(neginf=0.0)
    near = NEAR[out] * ((s * M + L).abs() <= NEAR[out] + 1).double()
    a, b = (torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)) for v in (d, lp))
    return lp.exp(), ref.EPS_SUM + ref.EPS * (2 * a + L.abs() + 2 * b + 8 + near)


def token_grad(z, s, y, g, ge, out):
    """(dlogits, bound of the kernel's error before its output rounding) in 64 bits."""
    d, L, lp = exact(z, s)
    p, rel = p_error(d, L, lp, z, s, out)
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    H = -(p * lp).sum(1, keepdim=True)
    g, ge = g.double()[:, None], ge.double()[:, None]
    dz = -s * p * (g + ge * (lp + H))
    dz.scatter_add_(1, y[:, None], s * g.expand_as(L))
    size = g.abs() + ge.abs() * (lp.abs() + H)
    bound = s * p * (rel * size + ge.abs() * (rel + ref.EPS_SUM * (2 + 2 * H)) + 4 * ref.EPS * size)
    bound = bound + s * 2e-38 * (1 + g.abs() + 200 * ge.abs())     # p flushed to zero
    bound.scatter_add_(1, y[:, None], s * g.abs().expand_as(L) * 2 * ref.EPS)
    empty = (z == -INF).all(1, keepdim=True)
    return dz.masked_fill(empty, 0.0), bound.masked_fill(empty, 0.0)


def distill_grad(z, s, ids, t, g, out):
    d, L, lp = exact(z, s)
    p, rel = p_error(d, L, lp, z, s, out)
    q, logq, _ = ref.teacher(ids, t, z.shape[1], s)
    g = g.double()[:, None]
    dz, bound = s * g * p, s * g.abs() * (p * (rel + 4 * ref.EPS) + 2e-38)
    at = ids.clamp(min=0)
    dz.scatter_add_(1, at, -s * g * q)
    bound.scatter_add_(1, at, s * g.abs() * q * ref.EPS * (16 + 4 * logq.abs()))
    none = (z == -INF).all(1, keepdim=True) | ~(q > 0).any(1, keepdim=True)
    return dz.masked_fill(none, 0.0), bound.masked_fill(none, 0.0)


def assert_grad_sums_to_zero(got, want, bound):
    ref.assert_grad(got, want, bound)
    dt = got.dtype
    room = (bound * (1 + ref.OUT_EPS[dt]) + want.abs() * ref.OUT_EPS[dt] + ref.OUT_TINY[dt]).sum(1)
    total = got.double().sum(1)
    assert bool((total.abs() <= room + 1e-12).all()), (total, room)


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("n,copies", [(1, 1), (40, 1), (5003, 1), (5003, 50), (40000, 1)])
def test_token_gradient_far_from_zero(rlk, dtype, out_dtype, temperature, n, copies):
    z, gen = far_rows(dtype, n, seed=n + 2)
    z = z.repeat(copies, 1)
    T, s = z.shape[0], 1.0 / temperature
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    g = torch.randn(T, generator=gen, device="cuda") * min(1.0, temperature)   # s g in the range of f16
    ge = torch.randn(T, generator=gen, device="cuda") * 0.1 * min(1.0, temperature)
    r = rlk.token_logprobs(z, y, temperature=temperature)
    d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, ge, temperature=temperature, out_dtype=out_dtype)
    assert_grad_sums_to_zero(d, *token_grad(z, s, y, g, ge, d.dtype))
    if out_dtype is None:                          # in place: the same bits
        z2 = z.clone()
        assert torch.equal(rlk.token_logprobs_bwd(z2, y, r.lse, r.entropy, g, ge, temperature=temperature, out=z2), d)
    d = rlk.token_logprobs_bwd(z, y, r.lse, None, g, temperature=temperature, out_dtype=out_dtype)
    assert_grad_sums_to_zero(d, *token_grad(z, s, y, g, torch.zeros_like(g), d.dtype))
    zero = torch.zeros_like(g)
    assert torch.count_nonzero(rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, zero, zero, temperature=temperature)) == 0


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("n,copies", [(1, 1), (40, 1), (5003, 1), (5003, 50), (40000, 1)])
def test_distillation_gradient_far_from_zero(rlk, dtype, out_dtype, temperature, n, copies):
    z, gen = far_rows(dtype, n, seed=n + 3)
    z = z.repeat(copies, 1)
    ids, t = near_teacher(z, 12, gen)
    g = torch.randn(z.shape[0], generator=gen, device="cuda") * min(1.0, temperature)
    kw = dict(temperature=temperature)
    _, lse = rlk.distill_topk_fwd(z, ids, t, **kw)
    d = rlk.distill_topk_bwd(z, ids, t, lse, g, out_dtype=out_dtype, **kw)
    assert_grad_sums_to_zero(d, *distill_grad(z, 1.0 / temperature, ids, t, g, d.dtype))
    assert torch.equal(rlk.distill_topk_fwd_bwd(z, ids, t, g, out_dtype=out_dtype, **kw)[2], d)
    if out_dtype is None:
        z2, z3 = z.clone(), z.clone()
        assert torch.equal(rlk.distill_topk_bwd(z2, ids, t, lse, g, out=z2, **kw), d)
        assert torch.equal(rlk.distill_topk_fwd_bwd(z3, ids, t, g, out=z3, **kw)[2], d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(3, 300001), (60, 151669), (700, 33001)])
def test_gradients_of_far_rows_among_others(rlk, dtype, T, n):
    """Long rows (two launches in the one-call step, many parts a row), misaligned, with columns beyond
    V_true, every third row far from zero."""
    V = n + 6
    gen = torch.Generator(device="cuda").manual_seed(T)
    buf = torch.full((T * (V + 1) + 3,), math.nan, dtype=dtype, device="cuda")
    z = buf[3:].view(T, V + 1)[:, :V]
    x = torch.randn((T, n), generator=gen, device="cuda") * 3
    x[::3] -= 5000.0
    x[::6] = torch.finfo(dtype).min
    z[:, :n] = x.to(dtype)
    del x
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    ids, t = near_teacher(z[:, :n], 9, gen)
    g = torch.rand(T, generator=gen, device="cuda") + 0.5
    r = rlk.token_logprobs(z, y, V_true=n)
    d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, g, V_true=n)
    _, lse, step = rlk.distill_topk_fwd_bwd(z, ids, t, g, V_true=n)
    dd = rlk.distill_topk_bwd(z, ids, t, lse, g, V_true=n)
    assert torch.equal(step, dd)
    assert torch.count_nonzero(d[:, n:]) == 0 and torch.count_nonzero(dd[:, n:]) == 0
    for a in range(0, T, 100):
        b = slice(a, min(T, a + 100))
        zb = z[b, :n]
        assert_grad_sums_to_zero(d[b, :n], *token_grad(zb, 1.0, y[b], g[b], g[b], dtype))
        assert_grad_sums_to_zero(dd[b, :n], *distill_grad(zb, 1.0, ids[b], t[b], g[b], dtype))
    out = z.clone()                                # rows V apart
    assert torch.equal(rlk.token_logprobs_bwd(out, y, r.lse, r.entropy, g, g, V_true=n, out=out), d)
    out = z.clone()
    assert torch.equal(rlk.distill_topk_bwd(out, ids, t, lse, g, V_true=n, out=out), dd)
    rlk.distill_topk_fwd_bwd(z, ids, t, g, V_true=n, out=z)
    assert torch.equal(z, dd)


@pytest.mark.parametrize("dtype", DTYPES)
def test_entropy_is_never_below_zero(rlk, dtype):
    """Not even by a rounding, in rows where one token takes all (its square root or logarithm may follow)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    for n in (1, 7, 5000):
        z = (torch.randn((600, n), generator=gen, device="cuda") * 5 +
             torch.randn((600, 1), generator=gen, device="cuda") * 50).to(dtype)
        for tau in (1.0, 0.7, 0.01, 1e-6, 3.0):
            assert float(rlk.token_logprobs(z, temperature=tau, top_k=1).entropy.min()) >= 0.0
            assert float(rlk.token_logprobs(z, temperature=tau).entropy.min()) >= 0.0


@pytest.mark.parametrize("dtype", DTYPES)
def test_checked_build_raises_no_flag_on_far_rows(rlk, dtype):
    """The reads of a row taken again stay inside it, misaligned, with columns beyond V_true, in place too."""
    from deterministic_token_logprob_gb300 import build
    build.build(debug_checks=True)
    n, V = 20003, 20010

    def run():
        rows, gen = far_rows(dtype, n, seed=5)
        T = rows.shape[0]
        z = torch.full((T, V + 1), math.nan, dtype=dtype, device="cuda")[:, 1:]
        z[:, :n] = rows
        y = torch.randint(0, n, (T,), generator=gen, device="cuda")
        ids, t = near_teacher(rows, 12, gen)
        g = torch.rand(T, generator=gen, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(V_true=n, err_flag=err)
        r = rlk.token_logprobs(z, y, top_k=7, **kw)
        out = [*r, rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, g, **kw), *rlk.distill_topk_fwd(z, ids, t, **kw),
               rlk.distill_topk_bwd(z, ids, t, r.lse, g, **kw), *rlk.distill_topk_fwd_bwd(z, ids, t, g, **kw)]
        out.append(rlk.distill_topk_bwd(z, ids, t, r.lse, g, out=z, **kw))
        torch.cuda.synchronize()
        return out, int(err)

    with rlk.library(build.DEBUG_LIB):
        assert rlk.debug_checks()
        checked, flag = run()
    plain, plain_flag = run()
    assert flag == 0 and plain_flag == 0
    for a, b in zip(checked, plain):
        assert torch.equal(a, b)
