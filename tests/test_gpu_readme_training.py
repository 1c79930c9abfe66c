"""README's step of a tied model, run as it stands: the gradients that it leaves are those of autograd in
64 bits, clipped."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_step_as_it_stands():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "rlk.clip_grad_norm(" in b)
    T, H, V, n = 40, 128, 700, 650
    gen = torch.Generator(device="cuda").manual_seed(0)
    W = (0.3 * torch.randn((V, H), generator=gen, device="cuda")).bfloat16()
    ids, y = (torch.randint(0, n, (T,), generator=gen, device="cuda") for _ in range(2))
    ids[3] = -1
    env = dict(rlk=rlk, W=W, w=1 + 0.1 * torch.randn(H, generator=gen, device="cuda"), b=torch.zeros(H, device="cuda"), ids=ids, y=y, s=11.0,
               V_true=n, g=torch.rand(T, generator=gen, device="cuda"))
    W64, w64 = W.double().requires_grad_(), env["w"].double().requires_grad_()
    exec(compile(block, "README.md", "exec"), env)
    x = torch.where((ids < 0)[:, None], 0.0, W64[ids.clamp(min=0)] * 11.0)
    h = x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w64
    logp = (h @ W64[:n].t()).log_softmax(1).gather(1, y[:, None])[:, 0]
    (logp * env["g"].double()).sum().backward()
    total = (W64.grad.square().sum() + w64.grad.square().sum()).sqrt()
    # bf16 rounds x, h, dz, dH and dx: five times 2^-8 at most, of values whose errors do not add up to more
    assert abs(float(env["norm"] / total) - 1) < 2e-2 and float(total) > 1
    for got, exact in ((env["dW"], W64.grad), (env["dw"], w64.grad)):
        assert float((got.double() - exact / total).norm() / (exact / total).norm()) < 2e-2
