"""Token log probabilities from logits (with rank, entropy and top alternatives), distillation
from a teacher's top logits, and their gradients, against plain 64-bit forms: element types, row
distances and alignments, odd and tiny sizes, masks that leave a row empty, ties, special values,
and the bitwise properties of the rows."""
import math

import pytest
import torch

import logits_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def make(T, V, n, dtype, seed, pad=0, offset=0, std=3.0):
    """Logits with rows V + pad apart that start `offset` elements into their buffer; the columns
    at and beyond n hold NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((T * (V + pad) + offset,), NAN, dtype=dtype, device="cuda")
    z = buf[offset:].view(T, V + pad)[:, :V]
    z[:, :n] = (torch.randn((T, n), generator=gen, device="cuda") * std).to(dtype)
    return z, gen


SIZES = [  # T, V, n, pad, offset
    (1, 1, 1, 0, 0),
    (3, 5, 4, 0, 0),
    (2, 9, 8, 0, 1),
    (5, 255, 255, 0, 0),
    (4, 257, 256, 3, 0),
    (3, 1023, 1023, 0, 3),
    (3, 1024, 1024, 0, 0),
    (2, 1025, 1025, 0, 0),
    (9, 2049, 2048, 7, 5),
    (17, 4096, 4090, 0, 0),
    (2, 33001, 33001, 0, 0),
    (7, 50257, 50257, 0, 0),
    (3, 151936, 151669, 128, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_scores(rlk, size, dtype):
    T, V, n, pad, offset = size
    z, gen = make(T, V, n, dtype, seed=V + T, pad=pad, offset=offset)
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k, tau in ((0, 1.0), (1, 0.7), (5, 1.0), (32, 2.0), (33, 1.0), (128, 1.3)):
        r = rlk.token_logprobs(z, y, top_k=k, V_true=n, temperature=tau, err_flag=err)
        ref.assert_scores(r, ref.scores(z, n, 1.0 / tau, y, k), z, n, 1.0 / tau)
    r = rlk.token_logprobs(z, top_k=3, V_true=n)
    assert r.logp is None and r.rank is None
    ref.assert_scores(r, ref.scores(z, n, 1.0, None, 3), z, n, 1.0)
    assert int(err) == 0


@pytest.mark.parametrize("T", [1, 2, 7, 31, 64, 150, 333, 700, 1300])
def test_scores_at_every_number_of_rows(rlk, T):
    z, gen = make(T, 8193, 8193, torch.bfloat16, seed=T)
    y = torch.randint(0, 8193, (T,), generator=gen, device="cuda")
    r = rlk.token_logprobs(z, y, top_k=20)
    ref.assert_scores(r, ref.scores(z, 8193, 1.0, y, 20), z, 8193, 1.0)


def test_largest_vocabulary(rlk):
    V = rlk.MAX_LOGITS_VOCAB
    z, gen = make(2, V, V - 3, torch.bfloat16, seed=1)
    y = torch.tensor([0, V - 4], device="cuda")
    r = rlk.token_logprobs(z, y, top_k=128, V_true=V - 3)
    ref.assert_scores(r, ref.scores(z, V - 3, 1.0, y, 128), z, V - 3, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_rows(rlk, dtype):
    """Rows beyond the shared memory that a step in one launch has, and beyond what a search for
    alternatives gets without asking."""
    V, n, K = 900000, 899999, 40
    z, gen = make(3, V, n, dtype, seed=30)
    y = torch.randint(0, n, (3,), generator=gen, device="cuda")
    r = rlk.token_logprobs(z, y, top_k=K, V_true=n)
    ref.assert_scores(r, ref.scores(z, n, 1.0, y, K), z, n, 1.0)
    ids, t = distill_inputs(3, n, K, gen)
    g = torch.rand(3, generator=gen, device="cuda")
    loss, lse, d = rlk.distill_topk_fwd_bwd(z, ids, t, g, V_true=n)
    want = ref.distill(z, n, V, 1.0, ids, t, g, lse)
    ref.assert_within(loss, want["loss"], ref.EPS_SUM + 64 * ref.EPS * want["loss_scale"], "loss")
    ref.assert_grad(d, want["dlogits"], want["bound"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_alternatives_that_crowd_or_tie(rlk, dtype):
    """The best columns side by side, in one lane's columns, or tied beyond what a bar can part: the
    second attempts of the search; and denormals, which order like other values."""
    n = 40000
    gen = torch.Generator(device="cuda").manual_seed(31)
    z = torch.randn((8, n), generator=gen, device="cuda").to(dtype)
    col = torch.arange(n, device="cuda")
    z[0, 20000:20300] = (20 + torch.arange(300, device="cuda") * 0.125).to(dtype)      # side by side
    z[1, (col % 256 < 8)] += 30                                                       # lane 0 of every leaf
    z[2] = (col % 3).to(dtype)                                                        # 13333 ties for the best
    z[3] = (-(col % 7).float()).to(dtype)                                             # ties of zero, then -1, ...
    z[4] = -4.0; z[4, 777] = -1.0; z[4, 30000:30050] = -2.0                           # ties below the best
    z[5] = torch.finfo(dtype).tiny * (torch.rand(n, generator=gen, device="cuda") - 0.5)
    z[6] = -float("inf"); z[6, ::1000] = 1.0                                          # 40 equal, nothing else
    z[7] = z[7].abs().neg()
    y = torch.randint(0, n, (8,), generator=gen, device="cuda")
    for k in (1, 20, 64, 128):
        r = rlk.token_logprobs(z, y, top_k=k)
        ref.assert_scores(r, ref.scores(z, n, 1.0, y, k), z, n, 1.0)
        for cut in (900, 5000):
            r = rlk.token_logprobs(z[:, 20000:20000 + cut], torch.zeros_like(y), top_k=k)
            part = z[:, 20000:20000 + cut]
            ref.assert_scores(r, ref.scores(part, cut, 1.0, torch.zeros_like(y), k), part, cut, 1.0)


def special_rows(dtype, n, gen):
    """Rows where masks, ties and special values go wrong, and a target for each."""
    big = torch.finfo(dtype).max
    r = (torch.randn((26, n), generator=gen, device="cuda") * 3).to(dtype)
    hide = torch.rand((26, n), generator=gen, device="cuda")
    y = torch.randint(0, n, (26,), generator=gen, device="cuda")
    r[0] = -INF                                   # empty
    r[1] = -INF; r[1, n // 2] = 2.0; y[1] = n // 2   # one left, chosen
    r[2] = -INF; r[2, n - 1] = -5.0; y[2] = 0        # one left, a masked token chosen
    r[3][hide[3] < 0.95] = -INF
    r[4][hide[4] < 0.95] = -big                   # masked by the type's lowest value
    r[5] = -big                                   # nothing but the lowest value: uniform
    r[6] = 1.5                                    # all equal: alternatives by index
    r[7] = torch.where(hide[7] < 0.5, 0.0, -0.0).to(dtype)  # zeros of both signs are equal
    r[8] = (r[8].float() / 2).round().to(dtype)   # many ties
    r[9] = torch.arange(n, device="cuda").to(dtype) / n          # ascending (with ties in 16 bits)
    r[10] = -torch.arange(n, device="cuda").to(dtype) / n        # descending
    r[11] = -INF; r[11, : min(n, 300)] = 1.0
    r[12, n // 3] = NAN
    r[13, n - 1] = INF
    r[14] = -INF; r[14, 0] = NAN
    r[15] = NAN
    r[16] = INF
    r[17, :] = -big; r[17, n // 4] = big          # differences beyond the type's range
    r[18] = 60.0; r[18, 0] = -60.0
    r[19][hide[19] < 0.5] = -INF; y[19] = int((r[19] == -INF).nonzero()[0]) if n > 8 else y[19]
    r[20] = -INF; r[20, max(0, n - 40):] = torch.arange(min(n, 40), device="cuda").to(dtype)  # clustered best
    y[21] = -1
    y[22] = n
    y[23] = -(1 << 40)
    r[24] = -INF; y[24] = n - 1
    r[25] = -0.0; y[25] = n - 1
    return r, y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 40, 1000, 5003, 20000])
def test_masks_ties_and_special_values(rlk, dtype, n):
    gen = torch.Generator(device="cuda").manual_seed(n)
    z, y = special_rows(dtype, n, gen)
    for k in (0, 8, 50, 128):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = rlk.token_logprobs(z, y, top_k=k, err_flag=err)
        ref.assert_scores(r, ref.scores(z, n, 1.0, y, k), z, n, 1.0)
        assert int(err) == rlk.RLK_FLAG_BAD_TARGET | rlk.RLK_FLAG_NONFINITE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [1e-6, 1.0])
def test_scaled_logits_at_the_edge_of_fp32(rlk, dtype, temperature):
    """s z is finite while s z log2(e) is not, in some leaves or in all of them."""
    n, edge = 5003, 3.0e38 * temperature
    gen = torch.Generator(device="cuda").manual_seed(n)
    z = torch.randn((10, n), generator=gen, device="cuda")
    y = torch.randint(0, n, (10,), generator=gen, device="cuda")
    z[0] = edge                                   # uniform at the edge
    z[1] = -edge
    z[2] = -edge; z[2, 7] = edge                  # one column takes all
    z[3] = -edge; z[3, ::100] = edge              # 51 columns share it
    z[4, :1024] = -edge                           # a leaf far down, the others ordinary
    z[5, 1024:2048] = -edge
    z[6, 4096:] = edge                            # the last leaf takes all
    z[7, 2000] = edge / 2                         # a maximum below the edge, its leaf's sums in range
    z[8] = edge / 2; z[8, 3000:] = edge
    z[9] = -INF; z[9, 50:60] = -edge              # masked besides
    z = z.to(dtype)
    for k in (0, 20):
        r = rlk.token_logprobs(z, y, top_k=k, temperature=temperature)
        ref.assert_scores(r, ref.scores(z, n, 1 / temperature, y, k), z, n, 1 / temperature)


def test_flags_name_their_cause(rlk):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = torch.zeros((2, 64), device="cuda")
    rlk.token_logprobs(z, torch.tensor([0, 64], device="cuda"), err_flag=err)
    assert int(err) == rlk.RLK_FLAG_BAD_TARGET
    err.zero_()
    z[1, 3] = NAN
    rlk.token_logprobs(z, torch.tensor([0, 1], device="cuda"), err_flag=err)
    assert int(err) == rlk.RLK_FLAG_NONFINITE
    err.zero_()
    rlk.token_logprobs(z, top_k=2, V_true=3, err_flag=err)  # the NaN lies beyond V_true
    assert int(err) == 0


def _grad_inputs(T, n, gen):
    g = torch.randn(T, generator=gen, device="cuda")
    ge = torch.randn(T, generator=gen, device="cuda") * 0.1
    if T > 2:
        g[1] = 0.0
        ge[1] = 0.0
        ge[2] = 0.0
    return g, ge


OUTS = [(torch.bfloat16, None), (torch.float16, None), (torch.float32, None), (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("size", SIZES)
def test_token_gradient(rlk, size, dtype, out_dtype):
    T, V, n, pad, offset = size
    z, gen = make(T, V, n, dtype, seed=V, pad=pad, offset=offset)
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    g, ge = _grad_inputs(T, n, gen)
    for tau in (1.0, 0.7):
        s = 1.0 / tau
        r = rlk.token_logprobs(z, y, V_true=n, temperature=tau)
        d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, ge, V_true=n, temperature=tau, out_dtype=out_dtype)
        assert d.shape == (T, V) and d.dtype == (out_dtype or dtype) and d.is_contiguous()
        ref.assert_grad(d, *ref.token_grad(z, n, V, s, y, r.lse, r.entropy, g, ge))
        d = rlk.token_logprobs_bwd(z, y, r.lse, None, g, V_true=n, temperature=tau, out_dtype=out_dtype)
        ref.assert_grad(d, *ref.token_grad(z, n, V, s, y, r.lse, r.entropy, g, torch.zeros_like(g)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_token_gradient_of_special_rows(rlk, dtype):
    n = 5003
    gen = torch.Generator(device="cuda").manual_seed(4)
    z, y = special_rows(dtype, n, gen)
    z, y = z[:17], y[:17]    # beyond: |s z| past the tolerance's range, and rows without a target
    z = torch.cat([z, z[:1]])
    y = torch.cat([y, torch.tensor([n], device="cuda")])
    g = torch.ones(18, device="cuda")
    r = rlk.token_logprobs(z, y)
    d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, g)
    zero = [0, 12, 13, 14, 15, 16, 17]   # empty, not finite, no target
    assert torch.count_nonzero(d[zero]) == 0
    keep = [i for i in range(17) if i not in zero and i not in (4, 5)]
    want, bound = ref.token_grad(z[keep].nan_to_num(nan=0.0, neginf=-INF), n, n, 1.0, y[keep], r.lse[keep],
                                 r.entropy[keep], g[keep], g[keep])
    ref.assert_grad(d[keep], want, bound)
    assert torch.isfinite(d).all()


def test_padding_rows_are_zero_whatever_they_hold(rlk):
    z = torch.full((3, 3000), NAN, device="cuda")
    z[1] = 0.0
    y = torch.zeros(3, dtype=torch.int64, device="cuda")
    g = torch.tensor([0.0, 1.0, 0.0], device="cuda")
    lse = torch.tensor([NAN, math.log(3000.0), INF], device="cuda")
    d = rlk.token_logprobs_bwd(z, y, lse, None, g)
    assert torch.count_nonzero(d[0]) == 0 and torch.count_nonzero(d[2]) == 0 and float(d[1, 0]) > 0.9
    ids = torch.zeros((3, 2), dtype=torch.int64, device="cuda")
    t = torch.zeros((3, 2), device="cuda")
    d = rlk.distill_topk_bwd(z, ids, t, lse, g)
    assert torch.count_nonzero(d[0]) == 0 and torch.count_nonzero(d[2]) == 0 and float(d[1, 0]) < -0.9


def distill_inputs(T, n, K, gen):
    ids = torch.randint(0, n, (T, K), generator=gen, device="cuda")     # ids come twice in small vocabularies
    t = torch.randn((T, K), generator=gen, device="cuda") * 4
    if K > 2:
        ids[::2, K - 1] = -1
        t[::3, 0] = -INF
    if T > 4:
        ids[4] = -1                 # no entries
        t[3] = -INF                 # none that counts
    return ids, t


@pytest.mark.parametrize("dtype,out_dtype", OUTS)
@pytest.mark.parametrize("size", SIZES)
def test_distillation(rlk, size, dtype, out_dtype):
    T, V, n, pad, offset = size
    z, gen = make(T, V, n, dtype, seed=V + 7, pad=pad, offset=offset)
    g, _ = _grad_inputs(T, n, gen)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for K, tau in ((1, 1.0), (7, 2.0), (32, 1.0), (100, 0.7), (128, 1.0)):
        s = 1.0 / tau
        ids, t = distill_inputs(T, n, K, gen)
        kw = dict(V_true=n, temperature=tau, err_flag=err)
        loss, lse = rlk.distill_topk_fwd(z, ids, t, **kw)
        want = ref.distill(z, n, V, s, ids, t, g, lse)
        x = z[:, :n].double() * s
        tol = ref.EPS_SUM + ref.EPS * (x.abs().max(1).values + want["lse"].abs())
        ref.assert_within(lse, want["lse"], tol, "lse")
        # q and log q: 2^-22.5 and the sum over K, then the products
        ref.assert_within(loss, want["loss"], tol + 32 * ref.EPS * want["loss_scale"], "loss")
        d = rlk.distill_topk_bwd(z, ids, t, lse, g, out_dtype=out_dtype, **kw)
        assert d.shape == (T, V) and d.dtype == (out_dtype or dtype)
        ref.assert_grad(d, want["dlogits"], want["bound"])
        # both at once: the same bits
        loss2, lse2, d2 = rlk.distill_topk_fwd_bwd(z, ids, t, g, out_dtype=out_dtype, **kw)
        assert torch.equal(loss2, loss) and torch.equal(lse2, lse) and torch.equal(d2, d)
    assert int(err) == 0


@pytest.mark.parametrize("T", [1, 2, 40, 160, 310, 1300])
def test_distillation_at_every_number_of_rows(rlk, T):
    n = 20011
    z, gen = make(T, n, n, torch.bfloat16, seed=T)
    ids, t = distill_inputs(T, n, 20, gen)
    g, _ = _grad_inputs(T, n, gen)
    loss, lse, d = rlk.distill_topk_fwd_bwd(z, ids, t, g)
    want = ref.distill(z, n, n, 1.0, ids, t, g, lse)
    ref.assert_within(loss, want["loss"], ref.EPS_SUM + 64 * ref.EPS * want["loss_scale"], "loss")
    ref.assert_grad(d, want["dlogits"], want["bound"])
    loss2, lse2 = rlk.distill_topk_fwd(z, ids, t)
    d2 = rlk.distill_topk_bwd(z, ids, t, lse2, g)
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse) and torch.equal(d2, d)


def test_distillation_special_rows(rlk):
    n, K = 4001, 6
    gen = torch.Generator(device="cuda").manual_seed(9)
    z = torch.randn((12, n), generator=gen, device="cuda")
    ids = torch.randint(0, n, (12, K), generator=gen, device="cuda")
    t = torch.randn((12, K), generator=gen, device="cuda")
    g = torch.ones(12, device="cuda")
    ids[0, 1] = n                     # outside
    ids[1, 0] = -2
    t[2, 3] = NAN
    t[3, 2] = INF
    t[4, 2] = NAN; ids[4, 2] = -1     # a value without an entry is never looked at
    z[5, 17] = NAN
    z[6, ids[6, 0]] = -INF            # the student masks a token that the teacher likes
    z[7] = -INF                       # the student has nothing
    ids[8] = ids[8, 0]                # one token in every place
    z[9] = -INF; z[9, ids[9]] = 1.0
    ids[10] = -1                      # the teacher has nothing
    z[11] = -INF; ids[11] = -1        # neither
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse, d = rlk.distill_topk_fwd_bwd(z, ids, t, g, err_flag=err)
    assert int(err) == rlk.RLK_FLAG_BAD_TARGET | rlk.RLK_FLAG_NONFINITE
    want = ref.distill(z, n, n, 1.0, ids, t, g, lse)
    ref.assert_within(loss, want["loss"], 1e-4, "loss")
    assert loss[[0, 1, 2, 3, 5]].isnan().all() and float(loss[6]) == INF and float(loss[7]) == INF
    assert float(loss[10]) == 0 and float(loss[11]) == 0
    assert torch.count_nonzero(d[[0, 1, 2, 3, 5, 7, 10, 11]]) == 0
    keep = [4, 6, 8, 9]
    ref.assert_grad(d[keep], want["dlogits"][keep], want["bound"][keep])
    loss2, lse2 = rlk.distill_topk_fwd(z, ids, t)
    d2 = rlk.distill_topk_bwd(z, ids, t, lse2, g)
    assert torch.equal(loss2.nan_to_num(nan=7.0), loss.nan_to_num(nan=7.0)) and torch.equal(d2, d)


@pytest.mark.parametrize("which", ["logp", "entropy", "loss"])
def test_gradient_against_differences(rlk, which):
    # central differences of the fp32 forward, step h: its error ~1e-6 / h from the forward's
    # rounding (|x| <= 16) and below h^2 / 6 from the third derivative (< 1)
    n, h = 37, 0.02
    gen = torch.Generator(device="cuda").manual_seed(12)
    z = torch.randn((1, n), generator=gen, device="cuda")
    y = torch.tensor([5], device="cuda")
    ids = torch.tensor([[5, 9, 9, -1, 30]], device="cuda")
    t = torch.randn((1, 5), generator=gen, device="cuda")
    one, zero = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    steps = torch.cat([z + h * torch.eye(n, device="cuda"), z - h * torch.eye(n, device="cuda")])
    for tau in (1.0, 0.8):
        if which == "loss":
            f, lse = rlk.distill_topk_fwd(steps, ids.expand(2 * n, -1).contiguous(), t.expand(2 * n, -1).contiguous(),
                                          temperature=tau)
            _, lse = rlk.distill_topk_fwd(z, ids, t, temperature=tau)
            d = rlk.distill_topk_bwd(z, ids, t, lse, one, temperature=tau)
        else:
            r = rlk.token_logprobs(steps, y.expand(2 * n).contiguous(), temperature=tau)
            f = getattr(r, which)
            r = rlk.token_logprobs(z, y, temperature=tau)
            d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, *((one, zero) if which == "logp" else (zero, one)),
                                       temperature=tau)
        diff = (f[:n] - f[n:]) / (2 * h)
        assert float((d[0] - diff).abs().max()) < 1e-6 / h + 4 * h * h / 6


def test_rows_do_not_depend_on_batch_position_or_alignment(rlk):
    """The bits of a row's outputs: alone, in batches of every launch shape, at another address."""
    n = 50257
    gen = torch.Generator(device="cuda").manual_seed(21)
    for dtype in DTYPES:
        row = (torch.randn(n, generator=gen, device="cuda") * 3).to(dtype)
        ids = torch.randint(0, n, (1, 9), generator=gen, device="cuda")
        t = torch.randn((1, 9), generator=gen, device="cuda")
        y = torch.tensor([777], device="cuda")
        one = torch.ones(1, device="cuda")
        a = rlk.token_logprobs(row[None], y, top_k=11)
        ga = rlk.token_logprobs_bwd(row[None], y, a.lse, a.entropy, one, one)
        da = rlk.distill_topk_fwd_bwd(row[None], ids, t, one)
        for T, at in ((2, 1), (5, 3), (40, 39), (170, 90), (400, 2), (1300, 1299)):
            z, _ = make(T, n, n, dtype, seed=T, pad=T % 7, offset=T % 3)
            z[at] = row
            yy = torch.randint(0, n, (T,), generator=gen, device="cuda")
            yy[at] = y
            r = rlk.token_logprobs(z, yy, top_k=11)
            for name in r._fields:
                assert torch.equal(getattr(r, name)[at], getattr(a, name)[0]), (name, dtype, T)
            ones = torch.ones(T, device="cuda")
            assert torch.equal(rlk.token_logprobs_bwd(z, yy, r.lse, r.entropy, ones, ones)[at], ga[0])
            dd = rlk.distill_topk_fwd_bwd(z, ids.expand(T, -1).contiguous(), t.expand(T, -1).contiguous(), ones)
            for u, v in zip(dd, da):
                assert torch.equal(u[at], v[0]), (dtype, T)


def test_offsets_beyond_32_bits(rlk):
    V, ld, T = 3001, 1 << 27, 20                      # the last row starts 2.5e9 elements in
    buf = torch.empty(ld * (T - 1) + V, dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((T, V), (ld, 1))
    small, gen = make(T, V, V, torch.bfloat16, seed=2)
    z.copy_(small)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    ids, t = distill_inputs(T, V, 5, gen)
    g, ge = _grad_inputs(T, V, gen)
    a, b = rlk.token_logprobs(z, y, top_k=4), rlk.token_logprobs(small, y, top_k=4)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    want = rlk.token_logprobs_bwd(small, y, b.lse, b.entropy, g, ge)
    assert torch.equal(rlk.token_logprobs_bwd(z, y, a.lse, a.entropy, g, ge), want)
    l0, _, d0 = rlk.distill_topk_fwd_bwd(small, ids, t, g)
    l1, _, d1 = rlk.distill_topk_fwd_bwd(z, ids, t, g, out=z)          # in place, rows far apart
    assert torch.equal(l0, l1) and torch.equal(d0, z) and d1.data_ptr() == z.data_ptr()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,pad,offset", [(4096, 0, 0), (5003, 0, 1), (9001, 5, 0)])
def test_gradient_in_place_of_the_logits(rlk, dtype, V, pad, offset):
    T, n = 33, V - 3
    z, gen = make(T, V, n, dtype, seed=3, pad=pad, offset=offset)
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    ids, t = distill_inputs(T, n, 12, gen)
    g, ge = _grad_inputs(T, n, gen)
    r = rlk.token_logprobs(z, y, V_true=n)
    want = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, ge, V_true=n)
    wantd = rlk.distill_topk_bwd(z, ids, t, r.lse, g, V_true=n)
    z1, _ = make(T, V, n, dtype, seed=3, pad=pad, offset=offset)
    assert rlk.token_logprobs_bwd(z1, y, r.lse, r.entropy, g, ge, V_true=n, out=z1) is z1
    assert torch.equal(z1, want)
    z2, _ = make(T, V, n, dtype, seed=3, pad=pad, offset=offset)
    rlk.distill_topk_bwd(z2, ids, t, r.lse, g, V_true=n, out=z2)
    assert torch.equal(z2, wantd)
    z3, _ = make(T, V, n, dtype, seed=3, pad=pad, offset=offset)
    rlk.distill_topk_fwd_bwd(z3, ids, t, g, V_true=n, out=z3)
    assert torch.equal(z3, wantd)


def test_outputs_beside_the_gradient_stay_untouched(rlk):
    T, V, n = 6, 3003, 2900
    z, gen = make(T, V, n, torch.float32, seed=5)
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    r = rlk.token_logprobs(z, y, V_true=n)
    one = torch.ones(T, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((T * 3100 + 9,), 7.0, dtype=dt, device="cuda")
        out = buf[5:5 + T * 3100].view(T, 3100)[:, 1:3050]             # wider than V, rows 3100 apart
        d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, one, one, V_true=n, out=out)
        assert d is out and torch.count_nonzero(out[:, n:]) == 0
        want = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, one, one, V_true=n, out_dtype=dt)
        assert torch.equal(out[:, :V], want)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_another_stream_and_graph_capture(rlk):
    T, V = 37, 20000
    z, gen = make(T, V, V, torch.bfloat16, seed=6)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    ids, t = distill_inputs(T, V, 16, gen)
    g, ge = _grad_inputs(T, V, gen)
    r = rlk.token_logprobs(z, y, top_k=6)
    d = rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, ge)
    step = rlk.distill_topk_fwd_bwd(z, ids, t, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2 = rlk.token_logprobs(z, y, top_k=6, stream=side)
    d2 = rlk.token_logprobs_bwd(z, y, r2.lse, r2.entropy, g, ge, stream=side)
    step2 = rlk.distill_topk_fwd_bwd(z, ids, t, g, stream=side)
    side.synchronize()
    for u, v in zip((*r, d, *step), (*r2, d2, *step2)):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3 = rlk.token_logprobs(z, y, top_k=6)
        d3 = rlk.token_logprobs_bwd(z, y, r3.lse, r3.entropy, g, ge)
        step3 = rlk.distill_topk_fwd_bwd(z, ids, t, g)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for u, v in zip((*r, d, *step), (*r3, d3, *step3)):
        assert torch.equal(u, v)


def test_autograd_gives_the_direct_calls_bits(rlk):
    T, V = 50, 6001
    z, gen = make(T, V, V, torch.bfloat16, seed=8)
    z = z.clone().requires_grad_()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    a, b = torch.randn(T, generator=gen, device="cuda"), torch.randn(T, generator=gen, device="cuda")
    logp, ent = rlk.token_logprobs_autograd(z, y, temperature=0.9)
    ((a * logp).sum() + (b * ent).sum()).backward()
    r = rlk.token_logprobs(z.detach(), y, temperature=0.9)
    assert torch.equal(logp, r.logp) and torch.equal(ent, r.entropy)
    assert torch.equal(z.grad, rlk.token_logprobs_bwd(z.detach(), y, r.lse, r.entropy, a, b, temperature=0.9))
    z.grad = None
    ids, t = distill_inputs(T, V, 10, gen)
    loss = rlk.distill_topk(z, ids, t, temperature=2.0)
    (a * loss).sum().backward()
    want = rlk.distill_topk_fwd_bwd(z.detach(), ids, t, a, temperature=2.0)
    assert torch.equal(loss, want[0]) and torch.equal(z.grad, want[2])


def test_gradient_feeds_the_products_of_the_staged_backward(rlk):
    """Saved logits -> dlogits in the dz workspace -> dH and dW, for the loss whose gradient the
    library's own backward knows: sum g logp."""
    T, H, V, n = 130, 256, 5100, 5003
    gen = torch.Generator(device="cuda").manual_seed(15)
    h = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    W = (torch.randn((V, H), generator=gen, device="cuda") * 0.05).bfloat16()
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    g = torch.randn(T, generator=gen, device="cuda")
    (logp, lse), z = rlk.linear_logp_fwd_save(h, W, y, n)
    r = rlk.token_logprobs(z, y, V_true=n)
    assert float((r.logp - logp).abs().max()) < 1e-5 and float((r.lse - lse).abs().max()) < 1e-5
    ws = torch.zeros(rlk.bwd_workspace_bytes(T, H, V), dtype=torch.uint8, device="cuda")
    rlk.token_logprobs_bwd(z, y, r.lse, None, g, V_true=n, out=rlk.bwd_dz_view(ws, T, V))
    dH, dW = rlk.linear_logp_bwd(h, W, y, r.lse, g, n, workspace=ws, stages=rlk.RLK_BWD_DH | rlk.RLK_BWD_DW)
    dH0, dW0 = rlk.linear_logp_bwd(h, W, y, lse, g, n)
    # the two dz round to bf16 from values that differ by fp32 rounding: few elements differ by a step
    assert float((dH.float() - dH0.float()).norm() / dH0.float().norm()) < 1e-3
    assert float((dW - dW0).norm() / dW0.norm()) < 1e-3


def test_empty_batch(rlk):
    z = torch.empty((0, 100), dtype=torch.float16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    f = torch.empty(0, device="cuda")
    r = rlk.token_logprobs(z, y, top_k=3)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 3)
    assert rlk.token_logprobs_bwd(z, y, f, f, f, f).shape == (0, 100)
    ids, t = torch.empty((0, 4), dtype=torch.int64, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, lse, d = rlk.distill_topk_fwd_bwd(z, ids, t, f)
    assert loss.shape == (0,) and d.shape == (0, 100)


def test_refusals(rlk):
    z = torch.zeros((4, 100), device="cuda")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    ids, t = torch.zeros((4, 5), dtype=torch.int64, device="cuda"), torch.zeros((4, 5), device="cuda")
    bad = [
        (ValueError, lambda: rlk.token_logprobs(z.cpu(), y)),
        (TypeError, lambda: rlk.token_logprobs(z.double(), y)),
        (ValueError, lambda: rlk.token_logprobs(z[0], y)),
        (ValueError, lambda: rlk.token_logprobs(z.t(), y)),
        (ValueError, lambda: rlk.token_logprobs(z[:1].expand(4, 100), y)),
        (TypeError, lambda: rlk.token_logprobs(z, y.int())),
        (ValueError, lambda: rlk.token_logprobs(z, y[:3])),
        (ValueError, lambda: rlk.token_logprobs(z, y, top_k=129)),
        (ValueError, lambda: rlk.token_logprobs(z, y, top_k=-1)),
        (ValueError, lambda: rlk.token_logprobs(z, y, V_true=101)),
        (ValueError, lambda: rlk.token_logprobs(z, y, V_true=0)),
        (rlk.RlkError, lambda: rlk.token_logprobs(z, y, temperature=0.0)),
        (rlk.RlkError, lambda: rlk.token_logprobs(z, y, temperature=-1.0)),
        (rlk.RlkError, lambda: rlk.token_logprobs(z, y, temperature=NAN)),
        (rlk.RlkError, lambda: rlk.token_logprobs(z, None, out=(f, None, f, f, None, None))),
        (ValueError, lambda: rlk.token_logprobs(z, y, out=(f, f))),
        (TypeError, lambda: rlk.token_logprobs(z, y, out=(f, f, f, f, None, None))),
        (ValueError, lambda: rlk.token_logprobs_bwd(z, y, f, None, f, f)),
        (rlk.RlkError, lambda: rlk.token_logprobs_bwd(z, y, f, f, f, out_dtype=torch.float16)),
        (ValueError, lambda: rlk.token_logprobs_bwd(z, y, f, f, f, out=z[:, :50])),
        (rlk.RlkError, lambda: rlk.token_logprobs_bwd(z[:3], y[:3], f[:3], f[:3], f[:3], out=z[1:])),  # overlap
        (TypeError, lambda: rlk.token_logprobs_bwd(z, y, f, f, f, out_dtype=torch.float64)),
        (ValueError, lambda: rlk.distill_topk_fwd(z, ids[:, :0], t[:, :0])),
        (ValueError, lambda: rlk.distill_topk_fwd(z, ids, t[:, :4])),
        (TypeError, lambda: rlk.distill_topk_fwd(z, ids, t.half())),
        (ValueError, lambda: rlk.distill_topk_fwd(z, ids.repeat(1, 40), t.repeat(1, 40))),
        (ValueError, lambda: rlk.distill_topk_bwd(z, ids, t, f[:2], f)),
        (ValueError, lambda: rlk.bwd_dz_view(torch.zeros(10, dtype=torch.uint8, device="cuda"), 4, 100)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
