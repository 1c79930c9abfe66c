"""README's example of the operators over logits, run as it stands: its gradients are those of the rows
that it scored."""
import ast
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_example_as_it_stands():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "rlk.token_logprobs(" in b)
    T, V, n, K = 9, 3000, 2900, 5
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    env = dict(rlk=rlk, torch=torch, logits=rand(T, V) * 3, V_true=n, g_logp=rand(T), g_entropy=rand(T), g=rand(T),
               y=torch.randint(0, n, (T,), generator=gen, device="cuda"), teacher=rand(T, K),
               ids=torch.randint(0, n, (T, K), generator=gen, device="cuda"))
    z = env["logits"].clone()
    scored = None
    for node in ast.parse(block).body:
        exec(compile(ast.Module([node], []), "README.md", "exec"), env)
        text = ast.unparse(node)
        if "rlk.token_logprobs(" in text:
            scored = node.value
        if "rlk.token_logprobs_bwd(" in text:  # against autograd of the same scores
            kw = eval(f"dict({', '.join(ast.unparse(k) for k in scored.keywords)})", env)
            x = z.clone().requires_grad_()
            logp = torch.log_softmax(x[:, :kw.get("V_true", V)].double() / kw.get("temperature", 1.0), 1)
            ent = -(logp.exp() * logp).sum(1)
            (env["g_logp"] * logp.gather(1, env["y"][:, None])[:, 0] + env["g_entropy"] * ent).sum().backward()
            assert float((env["r"].entropy - ent.detach()).abs().max()) < 1e-4
            # fp32 p: a few 1e-6 of |g| + |g_entropy| (|log p| + entropy), which stays below 60 here
            assert float((env["dz"] - x.grad).abs().max()) < 60 * 8e-6
            break
    else:
        raise AssertionError("no gradient of the scores in the example")
