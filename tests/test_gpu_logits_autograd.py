"""The operators over logits inside autograd: what it may and may not be told."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def inputs(T=6, V=300, K=4, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((T, V), generator=gen, device="cuda").to(dtype)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    ids = torch.randint(0, V, (T, K), generator=gen, device="cuda")
    return z, y, ids, torch.randn((T, K), generator=gen, device="cuda")


def test_second_derivatives_are_refused(rlk):
    """A penalty on the gradient must not lose its own derivative without a word."""
    z, y, ids, t = inputs()
    for f in (lambda x: rlk.token_logprobs_autograd(x, y)[0], lambda x: rlk.token_logprobs_autograd(x, y)[1],
              lambda x: rlk.distill_topk(x, ids, t)):
        x = z.clone().requires_grad_()
        (d,) = torch.autograd.grad(f(x).sum(), x, create_graph=True)
        (first,) = torch.autograd.grad(f(x).sum(), x)
        assert torch.equal(d.detach(), first)                    # the first derivative is as ever
        with pytest.raises(RuntimeError, match="differentiable once"):
            (x.sum() + (d * d).sum()).backward()


def test_what_a_call_overwrites_cannot_be_taken_for_what_was_saved(rlk):
    """A gradient written over logits that an earlier forward saved, and scores written over buffers
    that something saved, make that backward fail instead of giving other numbers."""
    z, y, ids, t = inputs()
    T = z.shape[0]
    g = torch.ones(T, device="cuda")
    r = rlk.token_logprobs(z, y)
    writes = [lambda x: rlk.token_logprobs_bwd(x, y, r.lse, r.entropy, g, g, out=x),
              lambda x: rlk.distill_topk_bwd(x, ids, t, r.lse, g, out=x),
              lambda x: rlk.distill_topk_fwd_bwd(x, ids, t, g, out=x),
              lambda x: rlk.distill_topk_fwd_bwd(x, ids, t, g, out=x, stream=torch.cuda.current_stream())]
    for write in writes:
        x = z.clone().requires_grad_()
        loss = rlk.distill_topk(x, ids, t).sum() + rlk.token_logprobs_autograd(x, y)[0].sum()
        write(x.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    for k, names in ((0, ("logp", "lse", "entropy")), (3, ("logp", "lse", "entropy", "top_logp"))):
        out = rlk.token_logprobs(z, y, top_k=k)
        for name in names:
            w = torch.ones_like(getattr(out, name), requires_grad=True)
            loss = (w * getattr(out, name)).sum()
            rlk.token_logprobs(z + 1, y, top_k=k, out=out)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()


def test_tensors_of_inference_mode_serve_as_outputs(rlk):
    z, y, ids, t = inputs()
    want = rlk.token_logprobs(z, y, top_k=3)
    g = torch.ones(z.shape[0], device="cuda")
    grad = rlk.token_logprobs_bwd(z, y, want.lse, None, g)
    with torch.inference_mode():
        buffers = [torch.empty_like(x) for x in want]
        d = torch.empty_like(z)
        rlk.token_logprobs(z, y, top_k=3, out=buffers)
    for x in buffers:
        x.detach()
    rlk.token_logprobs(z, y, top_k=3, out=buffers)
    assert all(torch.equal(a, b) for a, b in zip(buffers, want))
    assert torch.equal(rlk.token_logprobs_bwd(z, y, want.lse, None, g, out=d), grad)
