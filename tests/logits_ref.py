"""Plain 64-bit forms of the operators over logits (torch, elementary operations), and the
tolerances of the fp32 kernels against them, derived from their arithmetic.

Error of the row sum S (relative): ex2.approx 2^-22.5; rounding of the exponent |x| 2^-23 on a
term of weight 2^-|x|, at most 2^-23 log2(n) <= 20 x 1.2e-7 over the row; at most 16 + 5 + 32 + 5
additions in a chain, 58 x 6e-8. Together below EPS_SUM. s = fp32(1 / temperature) and each
final fused multiply-add add 2^-24 of the magnitudes they round.
"""
import math

import torch

EPS_SUM = 8e-6
EPS = 2.0 ** -23
OUT_EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
OUT_TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}  # half a denormal step / flush
NEG = -math.inf


def row_stats(z, n, s):
    """(x, lse, entropy, bad) of fp64 logits z[:, :n] at scale s; empty rows: lse -inf, entropy 0."""
    x = z[:, :n].double() * s
    bad = (x.isnan() | (x == math.inf)).any(1)
    m = x.max(1).values
    m0 = torch.where(m == NEG, torch.zeros_like(m), m)
    e = (x - m0[:, None]).exp()
    S = e.sum(1)
    lse = m0 + S.log()
    p = e / S[:, None]
    # about the maximum: lse itself has absorbed log S where |m| is the type's largest value
    ent = torch.where(S > 0, S.log() - torch.where(p > 0, p * (x - m0[:, None]), torch.zeros_like(p)).sum(1),
                      torch.zeros_like(S))
    nan = torch.full_like(lse, math.nan)
    return x, torch.where(bad, nan, lse), torch.where(bad, nan, ent), bad


def scores(z, n, s, y, k):
    """dict of logp, rank, lse, entropy, top_ids, top_logp in 64 bits."""
    x, lse, ent, bad = row_stats(z, n, s)
    zz = z[:, :n].double()
    T = z.shape[0]
    o = dict(lse=lse, entropy=ent)
    if y is not None:
        ok = (y >= 0) & (y < n)
        yc = torch.where(ok, y, torch.zeros_like(y))
        zy = zz.gather(1, yc[:, None])
        col = torch.arange(n, device=z.device)
        rank = 1 + ((zz > zy) | ((zz == zy) & (col < yc[:, None]))).sum(1)
        o["rank"] = torch.where(ok & ~bad, rank, torch.zeros_like(rank)).int()
        lp = torch.where(lse == NEG, lse, zy[:, 0] * s - lse)
        o["logp"] = torch.where(ok & ~bad, lp, torch.full_like(lp, math.nan))
    if k:
        order = torch.sort(zz + 0.0, dim=1, descending=True, stable=True)  # ties: lower index first
        kk = min(k, n)
        v, i = order.values[:, :kk], order.indices[:, :kk].clone()
        none = (v == NEG) | bad[:, None]
        i[none] = -1
        lp = v * s - lse[:, None]
        lp[none] = NEG
        lp[bad] = math.nan
        ids = torch.full((T, k), -1, dtype=torch.int64, device=z.device)
        top = torch.full((T, k), NEG, dtype=torch.float64, device=z.device)
        top[bad] = math.nan
        ids[:, :kk], top[:, :kk] = i, lp
        o["top_ids"], o["top_logp"] = ids, top
    return o


def token_grad(z, n, V, s, y, lse, ent, g, ge):
    """(dlogits [T, V], bound of the kernel's error before its output rounding), from the given
    fp32 lse and entropy."""
    T = z.shape[0]
    lse, ent, g, ge = (t.double()[:, None] for t in (lse, ent, g, ge))
    x = z[:, :n].double() * s
    d = x - torch.where(lse == NEG, torch.zeros_like(lse), lse)
    p = d.exp()
    pd = torch.where(p > 0, p * d, torch.zeros_like(p))
    dz = -s * (g * p + ge * (pd + p * ent))
    ok = (y >= 0) & (y < n)
    live = ok[:, None] & lse.isfinite() & ((g != 0) | (ge != 0))
    at = torch.where(ok, y, torch.zeros_like(y))[:, None]
    dz.scatter_add_(1, at, s * g)
    # p: |x| 2^-24 (s) + |d| (2^-24 + 2^-23) + 2^-22.5; then a few roundings of the products
    rel = EPS * (x.abs().clamp(max=1e4) + 2 * d.abs().clamp(max=1e4) + 8)
    bound = s * rel * ((g.abs() + ge.abs() * ent.abs()) * p + ge.abs() * pd.abs())
    bound.scatter_add_(1, at, s * g.abs() * 2 * EPS)
    dz, bound = (torch.where(live, t, torch.zeros_like(t)) for t in (dz, bound))
    pad = (0, V - n)
    return torch.nn.functional.pad(dz, pad), torch.nn.functional.pad(bound, pad)


def teacher(ids, t, n, s):
    """(q, log q, bad row) in 64 bits."""
    bad = ((ids < -1) | (ids >= n)).any(1)
    valid = (ids >= 0) & (ids < n)
    tt = torch.where(valid, t.double() * s, torch.full_like(t.double(), NEG))
    bad |= (tt.isnan() | (tt == math.inf)).any(1)
    m = tt.max(1, keepdim=True).values
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = (tt - m).exp()
    S = e.sum(1, keepdim=True)
    q = torch.where(S > 0, e / S, torch.zeros_like(e))
    logq = torch.where(q > 0, tt - m - S.log(), torch.zeros_like(q))
    return q, logq, bad


def distill(z, n, V, s, ids, t, g=None, lse32=None):
    """dict of loss, lse (and dlogits with its bound, from the given fp32 lse)."""
    x, lse, _, zbad = row_stats(z, n, s)
    q, logq, bad = teacher(ids, t, n, s)
    at = ids.clamp(min=0, max=n - 1)
    xk = x.gather(1, at)
    lp = torch.where(lse[:, None] == NEG, torch.full_like(xk, NEG), xk - lse[:, None])
    loss = torch.where(q > 0, q * (logq - lp), torch.zeros_like(q)).sum(1)
    nan = torch.full_like(loss, math.nan)
    scale = torch.where(q > 0, q * (logq.abs() + xk.abs() + lse.abs()[:, None]), torch.zeros_like(q)).sum(1)
    o = dict(loss=torch.where(bad | zbad, nan, loss), lse=lse, loss_scale=scale)
    if g is not None:
        l32, gg = lse32.double()[:, None], g.double()[:, None]
        some = (q > 0).any(1, keepdim=True) & ~bad[:, None] & l32.isfinite() & (gg != 0)
        d = x - torch.where(l32 == NEG, torch.zeros_like(l32), l32)
        p = d.exp()
        rel = EPS * (x.abs().clamp(max=1e4) + 2 * d.abs().clamp(max=1e4) + 8)
        dz, bound = s * gg * p, s * gg.abs() * p * rel
        dz.scatter_add_(1, at, -s * gg * q)
        # q: 2^-22.5, the sum over K <= 128 and its logarithm, |log q| 2^-23
        bound.scatter_add_(1, at, s * gg.abs() * q * EPS * (16 + logq.abs() * 4))
        dz, bound = (torch.where(some, v, torch.zeros_like(v)) for v in (dz, bound))
        pad = (0, V - n)
        o["dlogits"], o["bound"] = torch.nn.functional.pad(dz, pad), torch.nn.functional.pad(bound, pad)
    return o


def same_special(got, ref):
    """NaN and infinities stand in the same places (beyond the range of fp32 a value is infinite);
    returns the finite mask."""
    got, ref = got.float(), ref.float()
    assert torch.equal(got.isnan(), ref.isnan()), "NaN in other places"
    inf = ref.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], ref[inf]), "infinities in other places"
    return ref.isfinite()


def assert_within(got, ref, tol, what):
    ok = same_special(got, ref)
    err = (got.double() - ref.double()).abs()[ok]
    over = err - (tol.expand_as(ref)[ok] if isinstance(tol, torch.Tensor) else tol)
    assert err.numel() == 0 or float(over.max()) <= 0, f"{what}: error {float(err.max()):.3e}, over by {float(over.max()):.3e}"


def assert_scores(r, ref, z, n, s):
    """A TokenLogprobs against scores()."""
    x = z[:, :n].double() * s
    m = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).max(1).values  # largest finite magnitude
    lse0 = torch.where(ref["lse"].isfinite(), ref["lse"].abs(), torch.zeros_like(m))
    tol = EPS_SUM + EPS * (m + lse0)
    assert_within(r.lse, ref["lse"], tol, "lse")
    assert_within(r.entropy, ref["entropy"], EPS_SUM * (2 + 2 * ref["entropy"].nan_to_num().abs()), "entropy")
    if r.logp is not None:
        assert torch.equal(r.rank, ref["rank"]), "rank"
        assert_within(r.logp, ref["logp"], tol + EPS * ref["logp"].nan_to_num(neginf=0).abs(), "logp")
    if r.top_ids is not None:
        assert torch.equal(r.top_ids, ref["top_ids"]), "top_ids"
        assert_within(r.top_logp, ref["top_logp"],
                      tol[:, None] + EPS * ref["top_logp"].nan_to_num(neginf=0).abs(), "top_logp")


def assert_grad(got, ref, bound, what="dlogits"):
    dt = got.dtype
    assert_within(got, ref, bound + OUT_EPS[dt] * ref.abs() + OUT_TINY[dt] + bound * OUT_EPS[dt], what)
