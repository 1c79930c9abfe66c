"""Calls of the operators around the head that the other tests do not make."""
import pytest
import torch

import training_ref as ref
from test_gpu_training import PAIRS, norm_inputs, randn, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def test_lists_that_can_be_gone_through_once(rlk):
    """Gradients and results that come from a generator, on the current stream and on another one."""
    g = [torch.randn(1000, generator=rng(i), device="cuda") for i in range(3)]
    want = [torch.empty_like(x) for x in g]
    norm = rlk.clip_grad_norm(g, 1.0, out=want)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        out = [torch.empty_like(x) for x in g]
        torch.cuda.synchronize()
        assert torch.equal(rlk.clip_grad_norm((x for x in g), 1.0, out=(x for x in out), stream=stream), norm)
        assert torch.equal(rlk.grad_norm((x for x in g), stream=stream), norm)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T,H", [(7, 8193), (7, 12001), (7, 16383), (7, 16391), (3, 40003), (1100, 8200), (1100, 9001), (33, 4097)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_in_place_misaligned_and_wide(rlk, dtype, T, H):
    """The norm over x, and its gradient over dy or over x, on rows that start anywhere, beside their neighbours': the bits of the call into
    another tensor, within the bounds, and nothing between the rows is written."""
    for shift, pad in ((1, 1), (3, 0), (0, 5), (5, 2)):
        gen = rng(H + shift)
        x, w, b, dy = norm_inputs(gen, T, H, dtype, dtype, dtype)

        def odd(t):
            buf = torch.full((shift + T * (H + pad) + 3,), 9.0, dtype=dtype, device="cuda")
            rows = buf[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H]
            rows.copy_(t)
            return buf, rows

        for centered in (True, False):
            want = rlk.layer_norm_fwd(x, w, b, centered=centered)
            (wy, _, _), (ty, _, _) = ref.norm(x, w, b, 1e-5, centered)
            ref.close(want[0], wy, ref.rounded(wy, dtype, ty), "y")
            buf, rows = odd(x)
            got = rlk.layer_norm_fwd(rows, w, b, centered=centered, out=rows)
            assert got[0] is rows and all(p is q is None or torch.equal(p, q) for p, q in zip(got, want))
            rows.fill_(9.0)
            assert bool((buf == 9.0).all())
            _, mean, rstd = want
            grads = rlk.layer_norm_bwd(dy, x, w, mean, rstd)
            exact, tol = ref.norm_grad(dy, x, w, mean, rstd)
            for g, e, t in zip(grads, exact, tol):
                ref.close(g, e, ref.rounded(e, g.dtype, t))
            for over_x in (False, True):
                (xbuf, xrows), (dbuf, drows) = odd(x), odd(dy)
                to, buf = (xrows, xbuf) if over_x else (drows, dbuf)
                got = rlk.layer_norm_bwd(drows, xrows, w, mean, rstd, out=to)
                assert got[0] is to and all(torch.equal(p, q) for p, q in zip(got, grads))
                to.fill_(9.0)
                assert bool((buf == 9.0).all())


def test_rows_of_one_element_and_of_one_row(rlk):
    """Incoming gradients that autograd expands: strides of 0 where there is one row, one column or both."""
    for T, H in ((1, 1), (1, 8), (1, 300), (5, 1), (300, 1), (3, 8)):
        x = torch.randn((T, H), generator=rng(T + H), device="cuda", requires_grad=True)
        w = torch.randn(H, generator=rng(H), device="cuda", requires_grad=True)
        for f in (lambda: rlk.layer_norm(x, w, centered=False).sum(), lambda: rlk.layer_norm(x, w).mean(),
                  lambda: rlk.layer_norm(x, w)[:1].expand(4, H).sum(), lambda: (rlk.layer_norm(x, w, centered=False) * w).sum()):
            got = torch.autograd.grad(f(), (x, w))
            assert all(g.shape == t.shape and bool(g.isfinite().all()) for g, t in zip(got, (x, w)))
        table = torch.randn((T, H), generator=rng(3), device="cuda", requires_grad=True)
        (d,) = torch.autograd.grad(rlk.embedding(table, torch.zeros(T, dtype=torch.int64, device="cuda")).sum(), table)
        assert torch.equal(d[0], torch.full((H,), float(T), device="cuda")) and not d[1:].any()


def test_inference_mode(rlk):
    """Results into given tensors where there is no autograd."""
    with torch.inference_mode():
        x = torch.randn((6, 64), generator=rng(1), device="cuda")
        y, g, n = torch.empty_like(x), x.clone(), torch.empty((), device="cuda")
        assert rlk.layer_norm_fwd(x, out=y)[0] is y
        assert rlk.embedding_fwd(x, torch.tensor([5, 0], device="cuda"), out=y[:2]).shape == (2, 64)
        assert rlk.clip_grad_norm(g, 0.5, norm=n) is n
        assert abs(float(g.double().norm()) - 0.5) < 1e-6


def test_same_tensors_twice(rlk):
    """One token throughout, a gradient that is its own input's, a gradient listed twice, one tensor for weight and bias."""
    x = torch.randn((400, 64), generator=rng(2), device="cuda")
    same = torch.zeros(400, dtype=torch.int64, device="cuda")
    assert torch.equal(rlk.embedding_fwd(x, same), x[:1].expand(400, 64))
    want, tol = ref.table_grad(x, same, 400, 1.0, 0, 400, None)
    ref.close(rlk.embedding_bwd(x, same, 400), want, tol)
    w = torch.randn(64, generator=rng(3), device="cuda")
    y, mean, rstd = rlk.layer_norm_fwd(x, w, w)
    (wy, _, _), (ty, _, _) = ref.norm(x, w, w, 1e-5, True)
    ref.close(y, wy, ref.rounded(wy, torch.float32, ty))
    got = rlk.layer_norm_bwd(x, x, w, mean, rstd)
    want, tol = ref.norm_grad(x, x, w, mean, rstd)
    for g, e, t in zip(got, want, tol):
        ref.close(g, e, ref.rounded(e, g.dtype, t))
    n, rel = ref.total_norm([x, x])
    assert abs(float(rlk.grad_norm([x, x])) / n - 1) <= rel


def test_one_workspace_for_calls_in_turn(rlk):
    """One buffer for every call of a step on one stream, captured in two graphs that are replayed in turn."""
    T, H, V = 2000, 264, 500
    gen = rng(5)
    x, w, b, dy = norm_inputs(gen, T, H, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    ids = [torch.randint(0, V, (T,), generator=gen, device="cuda") for _ in range(2)]
    n = max(rlk.embedding_bwd_workspace_bytes(T, H), rlk.layer_norm_bwd_workspace_bytes(T, H), rlk.grad_norm_workspace_bytes(2))
    ws = torch.full((n,), 170, dtype=torch.uint8, device="cuda")
    _, mean, rstd = rlk.layer_norm_fwd(x, w, b)

    def step(i, **k):
        dx, dw, db = rlk.layer_norm_bwd(dy, x, w, mean, rstd, **k)
        dW = rlk.embedding_bwd(dx, ids[i], V, **k)
        return dx, dw, db, dW, rlk.clip_grad_norm([dW, dw], 0.1, **k)

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            got.append(step(i, workspace=ws))
    for _ in range(3):
        for i in (0, 1, 1, 0):
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))
