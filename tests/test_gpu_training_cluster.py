"""The table's gradient where its tokens are sorted by a cluster: every size of cluster, on an idle GPU and beside
work that keeps the SMs busy, so that the CTAs of a cluster start when they find room."""
import pytest
import torch

import training_ref as ref
from test_gpu_training import many_tokens, randn, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlk():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.mark.parametrize("T", [1024, 1025, 2049, 4100, 8193, 20001])   # 1, 2, 4, 8, 16 and 16 CTAs
@pytest.mark.parametrize("V", [300, 60000, 300000])                     # 1, 2 and 3 passes
def test_sort_beside_other_work(rlk, T, V):
    gen = rng(T)
    dout = randn(gen, T, 24, dtype=torch.bfloat16)
    ids = many_tokens(gen, T, V, "zipf")
    alone = rlk.embedding_bwd(dout, ids, V)
    want, tol = ref.table_grad(dout, ids, V, 1.0, 0, V, None)
    ref.close(alone, want, tol + ref.TINY[torch.float32])
    other = torch.cuda.Stream()
    a = torch.randn((2048, 2048), generator=gen, device="cuda", dtype=torch.float32).bfloat16()
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(other):
        for _ in range(60):
            a = (a @ a).clamp(-1, 1)
    for _ in range(8):
        got.append(rlk.embedding_bwd(dout, ids, V))
    torch.cuda.synchronize()
    assert all(torch.equal(g, alone) for g in got)


FIRST = """
import torch
import deterministic_token_logprob_gb300 as rlk
ids = torch.arange(5000, device="cuda") % 77
dout = torch.ones((5000, 16), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    dW = rlk.embedding_bwd(dout, ids, 100)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(dW, torch.bincount(ids, minlength=100).float()[:, None].expand(100, 16))
"""


def test_first_call_is_captured(rlk):
    """What the sort asks the device before its first launch may be asked while a graph is captured."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
