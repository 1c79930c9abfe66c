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
