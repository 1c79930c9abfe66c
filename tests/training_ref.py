"""Plain 64-bit forms of the operators around the head, and how far fp32 sums in a tree may be from them.

U is half a step of fp32 (2^-24), the most that one operation is off, relative to its result. A row's
sum goes through depth(H, S) additions at most: 4 for each of a slot's ceil(ceil(H / 8) / S) packs, 1 of even
and odd columns, 5 in a warp, 3 over the warps; S slots (at least), in the forward 32 up to 1024 columns, 64 up to 2048, 128 up to
4096 and 256 beyond, in the backward 32 up to 512, 64 up to 1024, 128 up to 2048. Every bound below counts roundings, times U, times the magnitudes that
they round; second orders are inside the few roundings that each count is rounded up by.
"""
import math

import torch

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half of the smallest value


def depth(H, forward):
    S = 32 * ((1 if H <= 1024 else 2 if H <= 2048 else 4 if H <= 4096 else 8) if forward else
              (1 if H <= 512 else 2 if H <= 1024 else 4 if H <= 2048 else 8))
    return 4 * -(-(-(-H // 8)) // S) + 9


def close(got, want, tol, name=""):
    """|got - want| <= tol, element by element, and NaN and infinities in the same places."""
    got = got.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    odd = ~want.isfinite()
    assert torch.equal(got[odd].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0), want[odd].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)), name
    over = torch.where(odd, -1.0, (got - want).abs() - tol)
    over = torch.where(over.isnan(), math.inf, over)
    if over.numel():
        i = int(over.argmax())
        assert float(over.max()) <= 0, (name, i, float(got.flatten()[i]), float(want.flatten()[i]))


def rounded(want, dtype, tol):
    """A value within tol of `want`, rounded once to dtype: how far it may be."""
    return tol + (want.abs() + tol) * STEP[dtype] + TINY[dtype]


# --------------------------------------------------------------------------- embedding


def lookup(table, ids, scale, start, V_true):
    """(x, tolerance before the last rounding)."""
    s = float(torch.tensor(scale, dtype=torch.float32))
    r = ids - start
    here = (ids >= 0) & (ids < V_true) & (r >= 0) & (r < table.shape[0])
    x = table[torch.where(here, r, 0)].double() * s
    x = torch.where(here[:, None], x, 0.0)
    x = torch.where(((ids < -1) | (ids >= V_true))[:, None], math.nan, x)
    return x, x.abs().nan_to_num() * U


def table_grad(dout, ids, V, scale, start, V_true, before):
    """(dW, tolerance): a term of n rows of one token goes through 16 additions in its run, 8 of its group's runs,
    one for each group of 128, and a product."""
    s = float(torch.tensor(scale, dtype=torch.float32))
    r = ids - start
    here = (ids >= 0) & (ids < V_true) & (r >= 0) & (r < V)
    d = dout[here].double()
    dW = torch.zeros((V, dout.shape[1]), dtype=torch.float64, device=dout.device)
    size = dW.clone()
    dW.index_add_(0, r[here], d)
    size.index_add_(0, r[here], d.abs())
    n = torch.bincount(r[here], minlength=V).double()[:, None]
    tol = (n.clamp(max=16) + (n / 16).ceil().clamp(max=8) + (n / 128).ceil() + 2) * U * size * abs(s)
    dW *= s
    if before is not None:
        dW = dW + before.double()
    return dW, tol + dW.abs() * U


# --------------------------------------------------------------------------- layer norm


def norm(x, w, b, eps, centered):
    """y, mean, rstd with their tolerances (y's before the last rounding)."""
    x = x.double()
    H = x.shape[1]
    m = x.mean(1, keepdim=True) if centered else torch.zeros_like(x[:, :1])
    d = x - m
    var = d.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    w = torch.ones(H, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(H, dtype=torch.float64, device=x.device) if b is None else b.double()
    y = d * r * w + b
    D, size = depth(H, True) + 5, d.abs().mean(1, keepdim=True)
    # x - m and the correction c: three roundings; c itself is a sum of differences over H. Before the correction the
    # mean is off by depth roundings of mean |x|, which the sum of differences sees in full and the square of which leaves
    # the variance to second order
    off = depth(H, True) * U * x.abs().mean(1, keepdim=True)
    td = 3 * U * (d.abs() + off) + D * U * (size + off)
    tvar = (D * U * (var + off * off) + 2 * size * D * U * (size + off)) * 2
    tr = r * (0.5 * tvar / (var + eps) + 4 * U)
    ty = w.abs() * (r * td + d.abs() * tr) + 3 * U * (d * r * w).abs() + U * y.abs()
    bad = ~x.isfinite().all(1)
    out = [torch.where(bad[:, None], math.nan, y), torch.where(bad, math.nan, m[:, 0]), torch.where(bad, math.nan, r[:, 0])]
    tol = [ty, D * U * (size + off)[:, 0] + 2 * U * m.abs()[:, 0], tr[:, 0]]
    return out, [torch.where(o.isfinite(), t, 0.0) for o, t in zip(out, tol)]


def norm_grad(dy, x, w, mean, rstd):
    """dx, dw, db with their tolerances (dx's before the last rounding), from given statistics."""
    T, H = x.shape
    dy = dy.double()
    r = rstd.double()[:, None]
    d = x.double() - (0.0 if mean is None else mean.double()[:, None])
    h = d * r                                       # two roundings
    w = torch.ones(H, dtype=torch.float64, device=x.device) if w is None else w.double()
    g = dy * w                                      # one
    c1 = g.mean(1, keepdim=True) if mean is not None else torch.zeros_like(r)
    c2 = (g * h).mean(1, keepdim=True)
    D = depth(H, False)
    t1 = (D + 3) * U * g.abs().mean(1, keepdim=True)
    t2 = (D + 6) * U * (g * h).abs().mean(1, keepdim=True)
    if mean is None:
        t1 = torch.zeros_like(t1)
    dx = r * (g - c1 - h * c2)
    tx = r * (t1 + h.abs() * t2 + U * (4 * g.abs() + 3 * c1.abs() + 6 * (h * c2).abs()))
    S = min(T, 304 * (8 if H <= 512 else 4 if H <= 1024 else 2 if H <= 2048 else 1))
    n = -(-T // S) + -(-S // 32) + 5 + 3            # additions in a strip, over strips of a group, over groups; a term's own
    dw, db = (dy * h).sum(0), dy.sum(0)
    return (dx, dw, db), (tx, n * U * (dy * h).abs().sum(0), n * U * dy.abs().sum(0))


# --------------------------------------------------------------------------- all gradients


def total_norm(grads):
    """(norm, relative tolerance): 16 products a thread and chunk added up one by one, even and odd apart, 17 roundings;
    one for each chunk of a share, 8 over a CTA's threads, 2 of the shares of a thread (which keep what they lose), 8 over threads
    again; half of all that through the root, and its own. A scale beside the norm's adds one more."""
    chunks = sum(-(-g.numel() * g.element_size() // 16384) for g in grads)
    n = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    return n, (0.5 * (-(-chunks // 912) + 36) + 1) * U
