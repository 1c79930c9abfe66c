"""One training loop over the operators on logits, as a trainer would chain them.

A teacher and a student are LM heads over the same hidden states. Each step
  1. scores the teacher's logits (`token_logprobs`): the sampled token's log probability and
     rank, the entropy, and the top alternatives, which are the distillation targets;
  2. computes the student's logits once (`linear_logp_fwd_save`, fp32 saved logits);
  3. distils (`distill_topk_fwd_bwd`): the loss and, straight into the dz workspace of the
     backward, its gradient with respect to the logits in bf16;
  4. turns that gradient into dH and dW with the library's tensor-core products
     (`linear_logp_bwd` with the stages RLK_BWD_DH | RLK_BWD_DW) and updates the student's head.

Run on a GPU: python examples/distill_from_logits.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import deterministic_token_logprob_gb300 as rlk  # noqa: E402


def run(steps: int = 20, T: int = 256, H: int = 256, V: int = 8192, V_true: int = 8000, K: int = 32,
        temperature: float = 2.0, lr: float = 0.1, verbose: bool = True):
    """Trains the student for `steps` steps; returns the mean loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    teacher_W = (randn(V, H) * 0.2).bfloat16()
    student = randn(V, H) * 0.02                        # fp32 master weights
    workspace = torch.empty(rlk.bwd_workspace_bytes(T, H, V), dtype=torch.uint8, device="cuda")
    dz = rlk.bwd_dz_view(workspace, T, V)               # what stage RLK_BWD_DZ would fill
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hidden = randn(T, H).bfloat16()
    losses = []
    for step in range(steps):
        y = torch.randint(0, V_true, (T,), generator=gen, device="cuda")
        (_, _), teacher_z = rlk.linear_logp_fwd_save(hidden, teacher_W, y, V_true)
        scored = rlk.token_logprobs(teacher_z, y, V_true=V_true, top_k=K, temperature=temperature, err_flag=err)
        W = student.bfloat16()
        (_, _), z = rlk.linear_logp_fwd_save(hidden, W, y, V_true)
        g = torch.full((T,), 1.0 / T, device="cuda")    # mean over the tokens
        # the log probabilities are at the temperature already; the operator divides by it again
        loss, lse, _ = rlk.distill_topk_fwd_bwd(z, scored.top_ids, scored.top_logp * temperature, g, V_true=V_true,
                                                temperature=temperature, out=dz, err_flag=err)
        dH, dW = rlk.linear_logp_bwd(hidden, W, y, lse, g, V_true, workspace=workspace,
                                     stages=rlk.RLK_BWD_DH | rlk.RLK_BWD_DW, err_flag=err)
        student -= lr * T * dW
        losses.append(loss.mean())
        if verbose:
            print(f"step {step:3d}  loss {float(losses[-1]):.4f}  teacher entropy {float(scored.entropy.mean()):.3f}  "
                  f"median rank of a random token {int(scored.rank.median())}  |dH| {float(dH.float().norm()):.2e}")
    assert int(err) == 0, f"device error flag {int(err)}"
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    run(ap.parse_args().steps)
