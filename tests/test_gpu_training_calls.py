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
