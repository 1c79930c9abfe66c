"""The operators over logits as they are used together, and in the debug-checks build."""
import importlib.util
import os

import pytest
import torch

import logits_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    build.build(debug_checks=True)
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def test_example_trains(rlk):
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "distill_from_logits.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.run(steps=12, T=128, H=128, V=2560, V_true=2500, K=16, verbose=False)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses  # full-batch gradient steps on a convex loss
    assert losses[-1] < 0.8 * losses[0]
    # the operators are deterministic: the same losses again
    assert m.run(steps=12, T=128, H=128, V=2560, V_true=2500, K=16, verbose=False) == losses


def test_distilled_gradients_of_the_head(rlk):
    """Saved logits -> loss and dz -> dH, dW against the formulas in 64 bits. dz is rounded to bf16
    once (2^-9 of each element, at random), dH once more: relative L2 below 1e-2 as elsewhere."""
    T, H, V, n, K = 200, 192, 3000, 2900, 20
    gen = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    W = (torch.randn((V, H), generator=gen, device="cuda") * 0.1).bfloat16()
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    ids = torch.randint(0, n, (T, K), generator=gen, device="cuda")
    t = torch.randn((T, K), generator=gen, device="cuda") * 2
    g = torch.rand(T, generator=gen, device="cuda")
    (_, _), z = rlk.linear_logp_fwd_save(h, W, y, n)
    ws = torch.empty(rlk.bwd_workspace_bytes(T, H, V), dtype=torch.uint8, device="cuda")
    loss, lse, dz = rlk.distill_topk_fwd_bwd(z, ids, t, g, V_true=n, out=rlk.bwd_dz_view(ws, T, V))
    dH, dW = rlk.linear_logp_bwd(h, W, y, lse, g, n, workspace=ws, stages=rlk.RLK_BWD_DH | rlk.RLK_BWD_DW)
    z64 = h.double() @ W.double().t()
    want = ref.distill(z64, n, V, 1.0, ids, t, g, torch.logsumexp(z64[:, :n], 1))
    assert float((loss - want["loss"]).abs().max()) < 2e-3
    for got, exact in ((dH, want["dlogits"] @ W.double()), (dW, want["dlogits"].t() @ h.double())):
        assert float((got.double() - exact).norm() / exact.norm()) < 1e-2


def _all(rlk, T, V, n, dtype, pad):
    gen = torch.Generator(device="cuda").manual_seed(T + V)
    z = (torch.randn((T, V + pad), generator=gen, device="cuda") * 3).to(dtype)[:, :V]
    z[0, : n // 2] = -float("inf")
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    ids = torch.randint(-1, n, (T, 37), generator=gen, device="cuda")
    t = torch.randn((T, 37), generator=gen, device="cuda")
    g = torch.randn(T, generator=gen, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(V_true=n, err_flag=err)
    out = []
    for k in (0, 7, 128):
        r = rlk.token_logprobs(z, y, top_k=k, **kw)
        out += [x for x in r if x is not None]
    out.append(rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, g, **kw))
    loss, lse = rlk.distill_topk_fwd(z, ids, t, **kw)
    out += [loss, lse, rlk.distill_topk_bwd(z, ids, t, lse, g, **kw), *rlk.distill_topk_fwd_bwd(z, ids, t, g, **kw)]
    if dtype == torch.float32:
        out.append(rlk.token_logprobs_bwd(z, y, r.lse, r.entropy, g, g, out_dtype=torch.bfloat16, **kw))
    torch.cuda.synchronize()
    return out, int(err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,V,n,pad", [(3, 9, 7, 0), (40, 5003, 5001, 2), (2, 50257, 50257, 0), (650, 2051, 2051, 0),
                                       (4, 151936, 151669, 0), (1200, 33000, 32999, 8)])
def test_checked_build_raises_no_flag_and_gives_the_same_bits(rlk, dtype, T, V, n, pad):
    from deterministic_token_logprob_gb300 import build
    with rlk.library(build.DEBUG_LIB):
        assert rlk.debug_checks()
        dbg, flag = _all(rlk, T, V, n, dtype, pad)
    rel, rel_flag = _all(rlk, T, V, n, dtype, pad)
    assert flag == 0 and rel_flag == 0
    for i, (a, b) in enumerate(zip(dbg, rel)):
        assert torch.equal(a, b), i
