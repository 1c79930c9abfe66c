"""The token log-probability and distillation operators over logits: the cases they are measured
at, their inputs, and their plain forms.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the
package's entry points. Two operators with their directions share the row statistics
(s = 1 / temperature, columns at or beyond v_true ignored). Token log probabilities:

  score         logp of the given token, its rank, lse, entropy, the k best tokens and their logp
  grad          gradient of sum_t g logp + g_entropy entropy with respect to the logits

and distillation:

  distill       KL divergence from a teacher's top-k distribution to the student's logits
  distill_grad  its gradient with respect to the student's logits
  distill_step  loss and gradient in one call (the token weights are known beforehand)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _case(name, op, T, V, v_true, dtype, k, temperature=1.0, masked=False, pad=0, out="same"):
    """k: alternatives (score) or teacher entries (distill*); pad: unused elements after each row;
    masked: rows come with most columns at -inf or the type's lowest value, some wholly; out: the
    gradient's type."""
    d = dict(op=op, T=T, V=V, v_true=v_true, dtype=dtype, k=k, temperature=temperature,
             masked=masked, pad=pad, out=out)
    if name:
        d["name"] = name
    return d


def listed():
    return [
        # One sequence being decoded: logp of the sampled token and the usual five alternatives.
        _case("score_one", "score", 1, 151936, 151669, "bf16", 5),
        # A decode step of a busy server, sampling at a temperature, 20 alternatives.
        _case("score_decode", "score", 64, 151936, 151669, "bf16", 20, temperature=0.7),
        # Constrained decoding: grammar masks, an odd vocabulary (rows at any 2-byte alignment).
        _case("score_masked", "score", 333, 50257, 50257, "f16", 8, masked=True),
        # Scoring a prompt with alternatives for every position.
        _case("score_prompt", "score", 1820, 151936, 151669, "bf16", 20),
        # A teacher's pass over saved fp32 logits (rows padded to 256 columns): its top 64.
        _case("score_teacher", "score", 4096, 151936, 151669, "f32", 64, pad=128),
        # Policy-gradient step of a small model on fp32 logits, with an entropy bonus.
        _case("grad_small", "grad", 64, 4096, 4096, "f32", 0),
        # The same for a batch with an odd vocabulary.
        _case("grad_odd", "grad", 796, 50257, 50257, "f16", 0, temperature=0.7),
        # The same at the framework's training size.
        _case("grad_train", "grad", 8192, 151936, 151669, "bf16", 0),
        # Evaluating a student: the distillation loss alone.
        _case("distill_eval", "distill", 512, 151936, 151669, "bf16", 64),
        # Backward of a loss computed before: fp32 logits, gradient in bf16 for the head's products.
        _case("distill_grad", "distill_grad", 1000, 32003, 32003, "f32", 32, temperature=2.0, out="bf16"),
        # A small student's training step.
        _case("distill_tiny", "distill_step", 16, 4096, 4096, "f32", 8, temperature=2.0),
        # A training step at the framework's training size.
        _case("distill_train", "distill_step", 8192, 151936, 151669, "bf16", 64),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "distill", "distill_grad", "distill_step"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    V = _log_uniform(rng, 1000, 151936)
    v_true = V - rng.choice([0, 0, rng.randrange(1, 300)])
    moved = BYTES[dtype] * V * (1 if op in ("score", "distill") else 2)
    T = _log_uniform(rng, 1, max(1, min(8192, (2 << 30) // moved)))
    k = 0 if op == "grad" else _log_uniform(rng, 1, 128)
    temperature = rng.choice([1.0, 1.0, 0.7, 1.3, 2.0])
    masked = rng.random() < 0.25
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    out = "bf16" if dtype == "f32" and op in ("grad", "distill_grad", "distill_step") and rng.random() < 0.5 else "same"
    return _case(None, op, T, V, v_true, dtype, k, temperature, masked, pad, out)


def prepare(case, seed):
    T, V, n, k = case["T"], case["V"], case["v_true"], case["k"]
    dt, dev = DTYPES[case["dtype"]], "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    # logits as language models give them: a broad bulk and a few likely tokens that stand out
    buf = torch.empty((T, V + case["pad"]), dtype=dt, device=dev)
    for a in range(0, T, 1024):
        rows = buf[a:a + 1024]
        rows.copy_(randn(*rows.shape).mul_(2.0))
    logits = buf[:, :V]
    # distinct tokens of each row, the first twelve the likely ones: one in each of `m` equal strips, rotated
    m = max(12, k)
    ids = (rand(T, 1) * n + (torch.arange(m, device=dev) + rand(T, m)) * (n // m)).long() % n
    likely = ids[:, :12]
    logits.scatter_(1, likely, (18 * rand(T, 1) - 1.5 * torch.arange(12, device=dev) + randn(T, 12)).to(dt))
    if case["masked"]:
        lowest = torch.finfo(dt).min
        for a in range(0, T, 1024):
            rows = logits[a:a + 1024]
            hide = rand(*rows.shape) < 0.95
            # every third row is masked by the type's lowest value, the others by -inf; every
            # eleventh row has nothing left
            kind = torch.arange(a, a + rows.shape[0], device=dev)[:, None]
            hide |= (kind % 11 == 5) & (kind % 3 != 0)
            rows.copy_(torch.where(hide, torch.where(kind % 3 == 0, lowest, -math.inf).to(dt), rows))
    state = {"case": case, "logits": logits, "V_true": n, "temperature": case["temperature"]}
    op = case["op"]
    s = 1.0 / case["temperature"]
    scale = 4096.0 if case["dtype"] == "f16" else 1.0   # f16 training scales its loss
    if op in ("score", "grad"):
        pick = (rand(T, 1) * 12).long()
        state["y"] = torch.where(rand(T) < 0.8, likely.gather(1, pick)[:, 0], (rand(T) * n).long())
    if op == "score":
        # the buffers that a serving loop keeps for the answers: logp, rank, lse, entropy, ids, their logp
        f32 = dict(dtype=torch.float32, device=dev)
        state["out"] = (torch.empty(T, **f32), torch.empty(T, dtype=torch.int32, device=dev), torch.empty(T, **f32),
                        torch.empty(T, **f32), torch.empty((T, k), dtype=torch.int64, device=dev),
                        torch.empty((T, k), **f32))
    if op in ("grad", "distill_grad"):  # the forward's statistics, which the program has kept
        lse, ent = [], []
        for a in range(0, T, 256):
            x = logits[a:a + 256, :n].double() * s
            l = x.logsumexp(1)
            p = (x - l.masked_fill(l == -math.inf, 0.0)[:, None]).exp()
            lse.append(l.float())
            ent.append(-torch.special.xlogy(p, p).sum(1).float())
        state["lse"], state["entropy"] = torch.cat(lse), torch.cat(ent)
    if op == "grad":
        state["g"] = randn(T) * scale / T               # advantages over the token count
        state["g_entropy"] = torch.full((T,), 0.01 * scale / T, device=dev)
    if op.startswith("distill"):
        # a teacher near the student: the likely tokens first, then others; some rows end in id -1
        ids = ids[:, :k].contiguous()
        teacher = 16 * rand(T, 1) - 8 * torch.log1p(torch.arange(k, device=dev)) + randn(T, k)
        if k > 2:
            ids[::7, -1] = -1
        if case["masked"]:                              # a teacher under the same mask
            teacher = torch.where(logits.gather(1, ids.clamp(min=0)) < -1e4, -math.inf, teacher)
        state["ids"], state["teacher"] = ids, teacher
        state["g"] = (0.5 + rand(T)) * scale / T
    if op in ("grad", "distill_grad", "distill_step"):
        state["out_dtype"] = dt if case["out"] == "same" else DTYPES[case["out"]]
    return state


def _softmax_parts(z, s):
    """(x - max, sum of exp, max) with max 0 for a row that has nothing left."""
    x = z.float() * s
    m = x.max(1, keepdim=True).values
    m = torch.where(m == -math.inf, 0.0, m)
    x = x - m
    return x, x.exp().sum(1, keepdim=True), m


def _widen(d, V, dtype):
    """The gradient over all V columns, zero at and beyond v_true, rounded once."""
    out = torch.zeros((d.shape[0], V), dtype=dtype, device=d.device)
    out[:, :d.shape[1]] = d
    return out


def _plain_score(S):
    z, y, s, k, n = S["logits"][:, :S["V_true"]], S["y"], 1.0 / S["temperature"], S["case"]["k"], S["V_true"]
    x, total, m = _softmax_parts(z, s)
    lse = m + total.log()
    e = x.exp()
    ent = torch.where(total > 0, total.log() - torch.where(e > 0, e * x, 0.0).sum(1, keepdim=True) / total, 0.0)
    del e, x
    zy = z.gather(1, y[:, None])
    logp = torch.where(lse == -math.inf, -math.inf, zy.float() * s - lse)
    col = torch.arange(n, device=z.device)
    rank = 1 + ((z > zy) | ((z == zy) & (col < y[:, None]))).sum(1)
    # unique whole-number keys in the order of (value, lower index first)
    bits = (z.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) + (n - 1 - col)
    kk = min(k, n)
    ids = n - 1 - (key.topk(kk, 1).values & 0xFFFFFFFF)
    top = z.gather(1, ids).float()
    ids = torch.where(top == -math.inf, -1, ids)
    top = torch.where(top == -math.inf, -math.inf, top * s - lse)
    if kk < k:
        ids = torch.nn.functional.pad(ids, (0, k - kk), value=-1)
        top = torch.nn.functional.pad(top, (0, k - kk), value=-math.inf)
    return {"logp": logp[:, 0], "rank": rank.int(), "lse": lse[:, 0], "entropy": ent[:, 0], "top_ids": ids, "top_logp": top}


def _plain_grad(S):
    z, y, s = S["logits"][:, :S["V_true"]], S["y"], 1.0 / S["temperature"]
    lse, ent, g, ge = (S[n][:, None] for n in ("lse", "entropy", "g", "g_entropy"))
    d = z.float() * s - torch.where(lse == -math.inf, 0.0, lse)
    p = d.exp()
    d = p * (-s * (g + ge * ent)) - s * ge * torch.where(p > 0, p * d, 0.0)
    d.scatter_add_(1, y[:, None], s * g)
    d = torch.where(lse == -math.inf, 0.0, d)
    return {"dlogits": _widen(d, S["case"]["V"], S["out_dtype"])}


def _teacher(S):
    """q over the valid entries (0 elsewhere) and log q (0 where q is 0)."""
    t = torch.where(S["ids"] < 0, -math.inf, S["teacher"].float() / S["temperature"])
    m = t.max(1, keepdim=True).values
    t = t - torch.where(m == -math.inf, 0.0, m)
    total = t.exp().sum(1, keepdim=True)
    logq = t - torch.where(total > 0, total, 1.0).log()
    q = torch.where(total > 0, logq.exp(), 0.0)
    return q, torch.where(q > 0, logq, 0.0)


def _plain_loss(S, q, logq, lse):
    zk = S["logits"].gather(1, S["ids"].clamp(min=0)).float() / S["temperature"]
    return torch.where(q > 0, q * (logq - torch.where(lse == -math.inf, -math.inf, zk - lse)), 0.0).sum(1)


def _plain_distill(S):
    q, logq = _teacher(S)
    _, total, m = _softmax_parts(S["logits"][:, :S["V_true"]], 1.0 / S["temperature"])
    lse = m + total.log()
    return {"loss": _plain_loss(S, q, logq, lse), "lse": lse[:, 0]}


def _plain_distill_grad(S, q, lse):
    s, g = 1.0 / S["temperature"], S["g"][:, None]
    some = (q > 0).any(1, keepdim=True)
    p = (S["logits"][:, :S["V_true"]].float() * s - torch.where(lse == -math.inf, 0.0, lse)).exp_()
    d = p.mul_(s * g)
    d.scatter_add_(1, S["ids"].clamp(min=0), -s * g * q)
    d = torch.where(some & (lse > -math.inf), d, 0.0)
    return _widen(d, S["case"]["V"], S["out_dtype"])


def _plain_step(S):
    q, logq = _teacher(S)
    _, total, m = _softmax_parts(S["logits"][:, :S["V_true"]], 1.0 / S["temperature"])
    lse = m + total.log()
    return {"loss": _plain_loss(S, q, logq, lse), "lse": lse[:, 0], "dlogits": _plain_distill_grad(S, q, lse)}


def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "score":
            return _plain_score(state)
        if op == "grad":
            return _plain_grad(state)
        if op == "distill":
            return _plain_distill(state)
        if op == "distill_grad":
            return {"dlogits": _plain_distill_grad(state, _teacher(state)[0], state["lse"][:, None])}
        return _plain_step(state)
    import deterministic_token_logprob_gb300 as rlk

    S, kw = state, dict(V_true=state["V_true"], temperature=state["temperature"])
    if op == "score":
        r = rlk.token_logprobs(S["logits"], S["y"], top_k=S["case"]["k"], out=S["out"], **kw)
        return {"logp": r.logp, "rank": r.rank, "lse": r.lse, "entropy": r.entropy, "top_ids": r.top_ids,
                "top_logp": r.top_logp}
    if op == "grad":
        return {"dlogits": rlk.token_logprobs_bwd(S["logits"], S["y"], S["lse"], S["entropy"], S["g"], S["g_entropy"],
                                                  out_dtype=S["out_dtype"], **kw)}
    if op == "distill":
        loss, lse = rlk.distill_topk_fwd(S["logits"], S["ids"], S["teacher"], **kw)
        return {"loss": loss, "lse": lse}
    if op == "distill_grad":
        return {"dlogits": rlk.distill_topk_bwd(S["logits"], S["ids"], S["teacher"], S["lse"], S["g"],
                                                out_dtype=S["out_dtype"], **kw)}
    loss, lse, dlogits = rlk.distill_topk_fwd_bwd(S["logits"], S["ids"], S["teacher"], S["g"],
                                                  out_dtype=S["out_dtype"], **kw)
    return {"loss": loss, "lse": lse, "dlogits": dlogits}


def work(case):
    T, V, n, k, e = case["T"], case["V"], case["v_true"], case["k"], BYTES[case["dtype"]]
    eo = e if case["out"] == "same" else BYTES[case["out"]]
    read, written, op = T * n * e, T * V * eo, case["op"]
    if op == "score":  # per row: y; logp, rank, lse, entropy, k ids and k logp
        return {"bytes": read + T * (8 + 16 + 12 * k), "flops": 6.0 * T * n}
    if op == "grad":   # per row: y, lse, entropy, g, g_entropy
        return {"bytes": read + written + T * 24, "flops": 6.0 * T * n}
    if op == "distill":
        return {"bytes": read + T * (12 * k + 8), "flops": 4.0 * T * n}
    if op == "distill_grad":
        return {"bytes": read + written + T * (12 * k + 8), "flops": 4.0 * T * n}
    return {"bytes": read + written + T * (12 * k + 12), "flops": 8.0 * T * n}


def exact(case, seed):
    """The definitions, row block by row block in 64 bits."""
    S = prepare(case, seed)
    T, V, n, k, s, op = case["T"], case["V"], case["v_true"], case["k"], 1.0 / case["temperature"], case["op"]
    parts = []
    for a in range(0, T, 256):
        r = slice(a, min(T, a + 256))
        z = S["logits"][r, :n].double()
        x = z * s
        row = torch.arange(z.shape[0], device=z.device)
        if op in ("grad", "distill_grad"):
            lse = S["lse"][r].double()
        else:
            lse = torch.logsumexp(x, 1)
        gone = lse == -math.inf
        lp = x - torch.where(gone, 0.0, lse)[:, None]   # log p (all -inf in an empty row)
        p = torch.exp(lp)
        o = {}
        if op == "score":
            o["lse"] = lse
            o["logp"] = lp[row, S["y"][r]]
            o["entropy"] = -torch.where(p > 0, p * lp, 0.0).sum(1)
            top = torch.topk(lp, min(k, n), 1).values
            o["top_logp"] = torch.nn.functional.pad(top, (0, k - top.shape[1]), value=-math.inf)
        elif op == "grad":
            g, ge, h = S["g"][r].double(), S["g_entropy"][r].double(), S["entropy"][r].double()
            d = -(g[:, None] * p) - ge[:, None] * torch.where(p > 0, p * (lp + h[:, None]), 0.0)
            d[row, S["y"][r]] += g
            d[gone] = 0.0
            o["dlogits"] = torch.nn.functional.pad(d * s, (0, V - n))
        else:
            ids, live = S["ids"][r], S["ids"][r] >= 0
            t = torch.where(live, S["teacher"][r].double() * s, -math.inf)
            q = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)   # a row without entries has none
            at = ids.clamp(min=0)
            if op != "distill_grad":
                o["lse"] = lse
                o["loss"] = (torch.special.xlogy(q, q) - torch.where(q > 0, q * lp.gather(1, at), 0.0)).sum(1)
            if op != "distill":
                d = p * (q.sum(1) > 0)[:, None]
                d.scatter_add_(1, at, -q)
                d[gone] = 0.0
                o["dlogits"] = torch.nn.functional.pad(d * (s * S["g"][r].double())[:, None], (0, V - n))
        parts.append(o)
    out = {name: torch.cat([q[name] for q in parts]) for name in parts[0]}
    if op == "score":
        out["rank"] = out["top_ids"] = None
    return out
