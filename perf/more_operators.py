"""The operators around the head in a training step -- embedding lookup, layer norm, each with its
gradient, and the global gradient norm with clipping: the cases they are measured at, their inputs,
and their plain forms.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the
package's entry points.

  embed       rows of the table by token, times a factor (token -1: padding, a zero row)
  embed_grad  the table's gradient in fp32: a new one (zero where no token points), or added to the
              head's dW, whose weight is the same table
  norm        (x - mean) rstd w + b over each row, or x rstd w about zero (centered False), with the
              statistics that the backward takes
  norm_grad   dx, and dw, db summed over the rows, from those statistics
  grad_norm   the 2-norm over many tensors
  clip        the same, and the tensors scaled so that it is at most max_norm
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _embed(name, op, T, H, V, dtype, scale=1.0, tied=False, words="zipf", padding=0.0, out="same"):
    """words: tokens as text has them (the r-th most frequent one in 1 / r of the cases), or spread
    evenly; padding: the share of tokens that are -1; tied: added to a gradient that is there."""
    d = dict(op=op, T=T, H=H, V=V, dtype=dtype, scale=scale, tied=tied, words=words, padding=padding, out=out)
    return dict(d, name=name) if name else d


def _norm(name, op, T, H, dtype, centered, out="same", weight="same", eps=1e-6):
    """weight: the weights' type (and the bias's, which centered rows have)."""
    d = dict(op=op, T=T, H=H, dtype=dtype, centered=centered, out=out, weight=weight, eps=eps)
    return dict(d, name=name) if name else d


def _clip(name, op, L, H, V, dtype, out="same"):
    """L layers of four [H, H] matrices and two [H] vectors; with V, a [V, H] table and another vector."""
    d = dict(op=op, L=L, H=H, V=V, dtype=dtype, out=out)
    return dict(d, name=name) if name else d


def listed():
    return [
        # A decode step of a busy server: one token of each of 64 sequences.
        _embed("embed_step", "embed", 64, 4096, 151936, "bf16"),
        # A training batch with padding, embeddings scaled by the root of the width.
        _embed("embed_train", "embed", 8192, 4096, 151936, "bf16", scale=64.0, padding=0.1),
        # The tiny model's step in fp32.
        _embed("embed_grad_tiny", "embed_grad", 64, 256, 4096, "f32"),
        # A table of its own at the framework's training size: most rows are zero.
        _embed("embed_grad_train", "embed_grad", 8192, 4096, 151936, "bf16", padding=0.1),
        # A table that is the head's weight as well: added to the head's dW.
        _embed("embed_grad_tied", "embed_grad", 16384, 2048, 151936, "bf16", scale=1.0, tied=True),
        # The norm before the head in a decode step.
        _norm("norm_step", "norm", 64, 4096, "bf16", False),
        # The same in training, from an fp32 residual stream to the head's bf16 operand.
        _norm("norm_train", "norm", 8192, 4096, "f32", True, out="bf16", weight="f32", eps=1e-5),
        # A small model of an odd width (rows at any 2-byte alignment).
        _norm("norm_grad_odd", "norm_grad", 796, 1001, "f16", True, eps=1e-5),
        # The backward at the framework's training size.
        _norm("norm_grad_train", "norm_grad", 8192, 4096, "bf16", False),
        # A small model's gradients, of odd sizes.
        _clip("clip_small", "clip", 2, 257, 4001, "f32"),
        # Many matrices in bf16, norm alone (a step that looks before it scales).
        _clip("grad_norm_layers", "grad_norm", 36, 1024, 0, "bf16"),
        # The head's dW and the final norm's weight.
        _clip("clip_head", "clip", 0, 4096, 151936, "f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly a multiple of 8, as hidden sizes are."""
    H = _log_uniform(rng, lo, hi)
    return H if rng.random() < 0.25 else -(-H // 8) * 8


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad", "grad_norm", "clip"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    out = "bf16" if dtype == "f32" and rng.random() < 0.4 else "same"
    if op in ("embed", "embed_grad"):
        H = _width(rng, 64, 8192)
        V = _log_uniform(rng, 500, min(151936, (500 << 20) // H))
        T = _log_uniform(rng, 1, min(32768, (128 << 20) // H))
        return _embed(None, op, T, H, V, dtype, rng.choice([1.0, 1.0, math.sqrt(H), 0.25]), op == "embed_grad" and rng.random() < 0.5,
                      rng.choice(["zipf", "zipf", "even"]), rng.choice([0.0, 0.0, rng.uniform(0.0, 0.6)]), out if op == "embed" else "same")
    if op in ("norm", "norm_grad"):
        H = _width(rng, 32, 16384)
        return _norm(None, op, _log_uniform(rng, 1, min(32768, (128 << 20) // H)), H, dtype, rng.random() < 0.5, out,
                     rng.choice(["same", "f32"]), rng.choice([1e-6, 1e-5]))
    H = _log_uniform(rng, 64, 2048)
    V = rng.choice([0, _log_uniform(rng, 500, min(151936, (200 << 20) // H))])
    return _clip(None, op, _log_uniform(rng, 1, max(1, min(64, (200 << 20) // (4 * H * H)))), H, V, dtype, out if op == "clip" else "same")


def _sizes(case):
    """Element counts of a clip case's tensors, in order."""
    H = case["H"]
    return [H * H, H, H * H, H * H, H, H * H] * case["L"] + ([case["V"] * H, H] if case["V"] else [])


def prepare(case, seed):
    dt, dev, op, H = DTYPES[case["dtype"]], "cuda", case["op"], case["H"]
    odt = dt if case["out"] == "same" else DTYPES[case["out"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def filled(rows, cols, dtype, factor):
        x = torch.empty((rows, cols), dtype=dtype, device=dev)
        for a in range(0, rows, 8192):
            part = x[a:a + 8192]
            part.copy_(randn(*part.shape).mul_(factor))
        return x

    if op in ("embed", "embed_grad"):
        T, V = case["T"], case["V"]
        if case["words"] == "zipf":  # the r-th most frequent token, and the tokens in no order of frequency
            ids = ((torch.exp(rand(T).double() * math.log(V)).long() - 1).clamp(0, V - 1) * 7919 + 13) % V
        else:
            ids = (rand(T).double() * V).long().clamp(0, V - 1)
        ids = torch.where(rand(T) < case["padding"], -1, ids)
        S = {"case": case, "ids": ids, "scale": case["scale"], "V": V, "out_dtype": odt}
        if op == "embed":
            S["table"] = filled(V, H, dt, 0.02)
        else:
            S["dout"] = filled(T, H, dt, 1.0 if case["dtype"] == "f16" else 1e-3)   # f16 training scales its loss
            S["dW"] = filled(V, H, torch.float32, 1e-3) if case["tied"] else None   # what the head's backward has left
        return S
    if op in ("norm", "norm_grad"):
        T = case["T"]
        wdt = dt if case["weight"] == "same" else DTYPES[case["weight"]]
        # a residual stream: rows of several sizes and offsets, and a few channels that stand out in all of them
        x = filled(T, H, dt, 1.0)
        loud = torch.where(rand(H) < 0.004, 30.0, 1.0)
        for a in range(0, T, 8192):
            r = x[a:a + 8192]
            r.copy_(r.float() * (0.5 + 2 * rand(r.shape[0], 1)) * loud + 0.3 * randn(r.shape[0], 1))
        S = {"case": case, "x": x, "w": (1 + 0.2 * randn(H)).to(wdt), "b": (0.1 * randn(H)).to(wdt) if case["centered"] else None,
             "eps": case["eps"], "out_dtype": odt}
        if op == "norm_grad":  # the forward's statistics, which the program has kept
            S["dy"] = filled(T, H, odt, 1.0 if case["dtype"] == "f16" else 1e-3)
            mean, rstd = [], []
            for a in range(0, T, 1024):
                z = x[a:a + 1024].double()
                m = z.mean(1, keepdim=True) if case["centered"] else torch.zeros_like(z[:, :1])
                mean.append(m[:, 0].float())
                rstd.append(((z - m).square().mean(1) + case["eps"]).rsqrt().float())
            S["mean"], S["rstd"] = torch.cat(mean) if case["centered"] else None, torch.cat(rstd)
        return S
    # gradients side by side in one buffer, each a view of it, as trainers keep them
    sizes = _sizes(case)
    total = sum(sizes)
    flat = torch.empty(total, dtype=dt, device=dev)
    for a in range(0, total, 1 << 26):
        part = flat[a:a + (1 << 26)]
        part.copy_(randn(part.numel()))
    grads = list(flat.split(sizes))
    loud = [math.exp(v) * (0.1 if case["dtype"] == "f16" else 1e-4) for v in (2 * randn(len(sizes))).clamp_(-4, 4).tolist()]
    for g, f in zip(grads, loud):
        g.mul_(f)
    S = {"case": case, "flat": flat, "grads": grads, "max_norm": 0.5 * math.sqrt(sum(n * f * f for n, f in zip(sizes, loud)))}
    if op == "clip":
        S["out_flat"] = torch.empty(total, dtype=odt, device=dev)
        S["out"] = list(S["out_flat"].split(sizes))
    return S


def _plain_embed(S):
    ids = S["ids"]
    x = S["table"].index_select(0, ids.clamp(min=0)).float() * S["scale"]
    return {"x": torch.where(ids[:, None] < 0, 0.0, x).to(S["out_dtype"])}


def _plain_embed_grad(S):
    live = S["ids"] >= 0
    g = torch.where(live[:, None], S["dout"].float() * S["scale"], 0.0)
    dW = S["dW"] if S["dW"] is not None else torch.zeros((S["V"], S["case"]["H"]), device=g.device)
    dW.index_add_(0, S["ids"].clamp(min=0), g)
    return {"dW": dW}


def _plain_norm(S):
    d = S["x"].float()
    mean = None
    if S["case"]["centered"]:
        mean = d.mean(1, keepdim=True)
        d = d - mean
    rstd = (d.square().mean(1, keepdim=True) + S["eps"]).rsqrt()
    y = d * rstd * S["w"].float()
    if mean is not None:
        y = y + S["b"].float()
    return {"y": y.to(S["out_dtype"]), "mean": None if mean is None else mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(S):
    rstd = S["rstd"][:, None]
    h = S["x"].float()
    if S["mean"] is not None:
        h = h - S["mean"][:, None]
    h = h * rstd
    dy = S["dy"].float()
    g = dy * S["w"].float()
    d = g - h * (g * h).mean(1, keepdim=True)
    if S["mean"] is not None:
        d = d - g.mean(1, keepdim=True)
    return {"dx": (d * rstd).to(S["x"].dtype), "dw": (dy * h).sum(0), "db": dy.sum(0) if S["mean"] is not None else None}


def _plain_clip(S):
    norm = S["flat"].float().square().sum(dtype=torch.float64).sqrt()
    if S["case"]["op"] == "grad_norm":
        return {"norm": norm.float()}
    factor = (S["max_norm"] / norm).clamp(max=1.0).float()
    S["out_flat"].copy_(S["flat"].float() * factor)
    return {"norm": norm.float(), "grads": S["out_flat"]}


def run(state):
    S, op = state, state["case"]["op"]
    if not own:
        if op == "embed":
            return _plain_embed(S)
        if op == "embed_grad":
            return _plain_embed_grad(S)
        if op == "norm":
            return _plain_norm(S)
        if op == "norm_grad":
            return _plain_norm_grad(S)
        return _plain_clip(S)
    import deterministic_token_logprob_gb300 as rlk

    if op == "embed":
        return {"x": rlk.embedding_fwd(S["table"], S["ids"], scale=S["scale"], out_dtype=S["out_dtype"])}
    if op == "embed_grad":
        return {"dW": rlk.embedding_bwd(S["dout"], S["ids"], S["V"], scale=S["scale"], out=S["dW"], accumulate=S["dW"] is not None)}
    if op == "norm":
        y, mean, rstd = rlk.layer_norm_fwd(S["x"], S["w"], S["b"], eps=S["eps"], centered=S["case"]["centered"], out_dtype=S["out_dtype"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = rlk.layer_norm_bwd(S["dy"], S["x"], S["w"], S["mean"], S["rstd"], want_db=S["mean"] is not None)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "grad_norm":
        return {"norm": rlk.grad_norm(S["grads"])}
    return {"norm": rlk.clip_grad_norm(S["grads"], S["max_norm"], out=S["out"]), "grads": S["out_flat"]}


def _rows_met(case):
    """How many rows of the table the tokens of such a case point at, on average."""
    T, V = case["T"] * (1 - case["padding"]), case["V"]
    if case["words"] != "zipf":
        return V * -math.expm1(T * math.log1p(-1 / V))
    met, r = 0.0, 1
    while r <= V:  # the r-th token has the share log((r + 1) / r) / log V; ranks in runs of up to 1 / 64 of their own size
        n = min(V - r + 1, 1 + r // 64)
        p = min(1.0 - 1e-12, math.log((r + n) / r) / n / math.log(V))
        met += n * -math.expm1(T * math.log1p(-p))
        r += n
    return met


def work(case):
    op, e, H = case["op"], BYTES[case["dtype"]], case["H"]
    eo = e if case["out"] == "same" else BYTES[case["out"]]
    if op in ("embed", "embed_grad"):
        T, V, met = case["T"], case["V"], _rows_met(case)
        if op == "embed":
            return {"bytes": T * (8 + H * eo) + met * H * e, "flops": 1.0 * T * H}
        live = T * (1 - case["padding"])
        written = 8 * met * H if case["tied"] else 4 * V * H
        return {"bytes": 8 * T + live * H * e + written, "flops": 2.0 * live * H}
    if op in ("norm", "norm_grad"):
        T, vectors = case["T"], 2 if case["centered"] else 1
        w = vectors * H * (e if case["weight"] == "same" else 4)
        if op == "norm":
            return {"bytes": T * H * (e + eo) + w + 4 * vectors * T, "flops": 8.0 * T * H}
        return {"bytes": T * H * (2 * e + eo) + w + 4 * vectors * (T + H), "flops": 14.0 * T * H}
    n = sum(_sizes(case))
    return {"bytes": n * e + (n * eo if op == "clip" else 0), "flops": 2.0 * n + (n if op == "clip" else 0)}


def exact(case, seed):
    """The definitions in 64 bits."""
    S, op = prepare(case, seed), case["op"]
    if op == "embed":
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        live = S["ids"] >= 0
        out[live] = S["table"][S["ids"][live]].double() * case["scale"]
        return {"x": out}
    if op == "embed_grad":
        dW = torch.zeros((case["V"], case["H"]), dtype=torch.float64, device="cuda")
        for a in range(0, case["T"], 1024):
            live = S["ids"][a:a + 1024] >= 0
            dW.index_add_(0, S["ids"][a:a + 1024][live], S["dout"][a:a + 1024][live].double())
        dW *= case["scale"]
        if S["dW"] is not None:
            dW += S["dW"]
        return {"dW": dW}
    if op in ("norm", "norm_grad"):
        w, parts = S["w"].double(), []
        for a in range(0, case["T"], 1024):
            r = slice(a, a + 1024)
            x, o = S["x"][r].double(), {}
            if op == "norm":
                var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
                if not case["centered"]:
                    var, mean = (x * x).sum(1, keepdim=True) / case["H"], torch.zeros_like(mean)
                o["rstd"] = 1 / torch.sqrt(var[:, 0] + case["eps"])
                o["y"] = (x - mean) * w * o["rstd"][:, None]
                if case["centered"]:
                    o["mean"], o["y"] = mean[:, 0], o["y"] + S["b"].double()
            else:
                rstd, dy = S["rstd"][r].double()[:, None], S["dy"][r].double()
                if case["centered"]:
                    x = x - S["mean"][r].double()[:, None]
                h = x * rstd
                dh = dy * w
                o["dx"] = rstd * (dh - h * torch.einsum("th,th->t", dh, h)[:, None] / case["H"])
                if case["centered"]:
                    o["dx"] -= rstd * dh.sum(1, keepdim=True) / case["H"]
                    o["db"] = dy.sum(0, keepdim=True)
                o["dw"] = (dy * h).sum(0, keepdim=True)
            parts.append(o)
        out = {n: torch.cat([q[n] for q in parts]) for n in parts[0]}
        for n in ("dw", "db"):
            if n in out:
                out[n] = out[n].sum(0)
        return {**({"mean": None} if op == "norm" else {"db": None}), **out}
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for a in range(0, S["flat"].numel(), 1 << 26):
        part = S["flat"][a:a + (1 << 26)].double()
        total += torch.dot(part, part)
    norm = torch.sqrt(total)
    if op == "grad_norm":
        return {"norm": norm}
    return {"norm": norm, "grads": S["flat"].double() * min(1.0, S["max_norm"] / norm.item())}
