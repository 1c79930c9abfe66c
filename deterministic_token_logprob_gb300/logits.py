"""Operators over logits that already exist: token log probabilities with entropy and top
alternatives (:func:`token_logprobs`), their gradient (:func:`token_logprobs_bwd`), and
distillation from a teacher's top logits (:func:`distill_topk_fwd`, :func:`distill_topk_bwd`,
:func:`distill_topk_fwd_bwd`).

Argument marshalling around the C entry points of the same names (include/rlk.h states their
mathematics, special rows and errors); all arithmetic runs in the library's CUDA kernels.
``logits`` is a [T, V] CUDA tensor of bfloat16, float16 or float32 whose rows are contiguous
(stride(1) == 1; stride(0) is free, so a slice of a wider buffer serves), and ``V_true``
defaults to V. Work is enqueued on ``stream`` (default: the current stream of the logits'
device); with a ``stream`` given, outputs are allocated on it and the inputs are recorded as
used there.

:func:`token_logprobs_autograd` and :func:`distill_topk` are the autograd forms.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from ._binding import _check, _load

RLK_DTYPE_BF16 = 0
RLK_DTYPE_F16 = 1
RLK_DTYPE_F32 = 2
MAX_TOP_K = 128
MAX_LOGITS_VOCAB = 1 << 20

_DTYPES = {torch.bfloat16: RLK_DTYPE_BF16, torch.float16: RLK_DTYPE_F16, torch.float32: RLK_DTYPE_F32}


class TokenLogprobs(NamedTuple):
    """Per row: the token's log probability (fp32) and rank (int32, 1 = most likely), lse and
    entropy (fp32), and the top_k best tokens (int64 [T, top_k], -1 where there is none) with
    their log probabilities (fp32 [T, top_k]). Without targets logp and rank are None; with
    top_k = 0 the last two are."""
    logp: Optional[torch.Tensor]
    rank: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


# The current device and stream without building torch objects: a small call (one token, or a small
# model's step) is bounded by its work on the host.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
# Tells autograd that tensors have been written to (a kernel's writes are not its to see).
_written = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int, int, int, int]:
    """Checks a [T, V] CUDA tensor with contiguous rows; (T, V, row distance, dtype code, device index)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {[str(d) for d in _DTYPES]}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(shape)}")
    T, V = shape
    ld, inner = t.stride()
    if inner != 1 and V > 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    if ld < V:
        if T > 1:
            raise ValueError(f"{name} must not have overlapping rows")
        ld = V  # the stride of a single row says nothing
    return T, V, ld, code, dev


def _per_row(t, name: str, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this dtype, shape and device index."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _flag(err_flag, dev):
    return None if err_flag is None else _per_row(err_flag, "err_flag", torch.int32, (1,), dev)


def _away(stream, dev) -> bool:
    """Whether a call has to change the current stream or device first (see _elsewhere)."""
    return stream is not None or dev != _current_device()


@contextlib.contextmanager
def _elsewhere(stream, device, tensors):
    """Makes `device` and `stream` current, so that outputs belong to that stream, and records
    `tensors` as used there."""
    if stream is not None and stream.device_index != device:
        raise ValueError(f"stream must be one of cuda:{device}, got one of {stream.device}")
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        with torch.cuda.stream(stream):
            yield
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _true_vocab(V_true: Optional[int], V: int) -> int:
    V_true = V if V_true is None else int(V_true)
    if not 0 < V_true <= V:
        raise ValueError(f"V_true must be in 1 .. {V}, got {V_true}")
    return V_true


def token_logprobs(logits: torch.Tensor, y: Optional[torch.Tensor] = None, *, top_k: int = 0,
                   V_true: Optional[int] = None, temperature: float = 1.0,
                   out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                   err_flag: Optional[torch.Tensor] = None, stream=None) -> TokenLogprobs:
    """rlk_token_logprobs: the log probability and rank of each row's token y (int64 [T]), lse,
    entropy and the top_k alternatives of softmax(logits / temperature).

    `out` supplies the six output tensors in the order of :class:`TokenLogprobs` (a serving loop
    keeps them between steps); None in a place leaves that output out."""
    T, V, ld, code, dev = _rows(logits, "logits")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (logits, y, err_flag, *(out or ()))):
            return token_logprobs(logits, y, top_k=top_k, V_true=V_true, temperature=temperature, out=out,
                                  err_flag=err_flag)
    V_true = _true_vocab(V_true, V)
    if not 0 <= top_k <= MAX_TOP_K:
        raise ValueError(f"top_k must be in 0 .. {MAX_TOP_K}, got {top_k}")
    rows, i32, i64, f32 = (T,), torch.int32, torch.int64, torch.float32
    py = None if y is None else _per_row(y, "y", i64, rows, dev)
    if out is None:
        on = logits.device
        r = TokenLogprobs(None if y is None else torch.empty(T, dtype=f32, device=on),
                          None if y is None else torch.empty(T, dtype=i32, device=on),
                          torch.empty(T, dtype=f32, device=on), torch.empty(T, dtype=f32, device=on),
                          torch.empty((T, top_k), dtype=i64, device=on) if top_k else None,
                          torch.empty((T, top_k), dtype=f32, device=on) if top_k else None)
    elif len(out) != 6:
        raise ValueError("out must hold six tensors (or None): logp, rank, lse, entropy, top_ids, top_logp")
    else:
        r = TokenLogprobs(*out)
    logp, rank, lse, entropy, ids, top = r
    st = _load().rlk_token_logprobs(
        logits.data_ptr(), code, T, ld, V_true, temperature, py, top_k,
        None if logp is None else _per_row(logp, "logp", f32, rows, dev),
        None if rank is None else _per_row(rank, "rank", i32, rows, dev),
        None if lse is None else _per_row(lse, "lse", f32, rows, dev),
        None if entropy is None else _per_row(entropy, "entropy", f32, rows, dev),
        None if ids is None else _per_row(ids, "top_ids", i64, (T, top_k), dev),
        None if top is None else _per_row(top, "top_logp", f32, (T, top_k), dev),
        _flag(err_flag, dev), _raw_stream(dev))
    if st:
        _check("rlk_token_logprobs", st)
    if out is not None:
        some = logp is None or rank is None or lse is None or entropy is None or ids is None or top is None
        _written([x for x in r if x is not None] if some else r)
    return r


def _gradient(logits, T, V, out, out_dtype):
    """The dlogits tensor to fill -- `out` ([T, at least V], rows contiguous) or a new [T, V] one --
    and its C arguments."""
    if out is None:
        dtype = out_dtype or logits.dtype
        code = _DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"out_dtype must be one of {[str(d) for d in _DTYPES]}, got {dtype}")
        d = torch.empty((T, V), dtype=dtype, device=logits.device)
        return d, (d.data_ptr(), code, V, max(V, 1))
    oT, oV, old, code, dev = _rows(out, "out")
    if oT != T or oV < V:
        raise ValueError(f"out must have {T} rows of at least {V} columns, got {tuple(out.shape)}")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    if dev != logits.get_device():
        raise ValueError(f"out must be on {logits.device}, got {out.device}")
    return out, (out.data_ptr(), code, oV, old)


def token_logprobs_bwd(logits: torch.Tensor, y: torch.Tensor, lse: torch.Tensor,
                       entropy: Optional[torch.Tensor], g_logp: torch.Tensor,
                       g_entropy: Optional[torch.Tensor] = None, *, V_true: Optional[int] = None,
                       temperature: float = 1.0, out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None,
                       err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rlk_token_logprobs_bwd -> dlogits of sum_t (g_logp logp + g_entropy entropy), from the
    forward's lse and entropy. The result has the logits' shape and type (or out_dtype: bfloat16
    for float32 logits); `out` supplies it, the logits themselves included (autograd takes it for
    modified in place)."""
    T, V, ld, code, dev = _rows(logits, "logits")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (logits, y, lse, entropy, g_logp, g_entropy, out, err_flag)):
            return token_logprobs_bwd(logits, y, lse, entropy, g_logp, g_entropy, V_true=V_true,
                                      temperature=temperature, out=out, out_dtype=out_dtype, err_flag=err_flag)
    rows, f32 = (T,), torch.float32
    if g_entropy is not None and entropy is None:
        raise ValueError("g_entropy needs the forward's entropy")
    p = (_per_row(y, "y", torch.int64, rows, dev), _per_row(lse, "lse", f32, rows, dev),
         None if entropy is None else _per_row(entropy, "entropy", f32, rows, dev),
         _per_row(g_logp, "g_logp", f32, rows, dev),
         None if g_entropy is None else _per_row(g_entropy, "g_entropy", f32, rows, dev))
    V_true = _true_vocab(V_true, V)
    dlogits, d = _gradient(logits, T, V, out, out_dtype)
    st = _load().rlk_token_logprobs_bwd(logits.data_ptr(), code, T, ld, V_true, temperature, *p, *d,
                                        _flag(err_flag, dev), _raw_stream(dev))
    if st:
        _check("rlk_token_logprobs_bwd", st)
    if out is not None:
        _written((out,))
    return dlogits


def _teacher(ids, teacher, T, dev):
    shape = ids.shape if isinstance(ids, torch.Tensor) else ()
    if len(shape) != 2:
        raise ValueError("ids must be an int64 [T, K] tensor")
    K = shape[1]
    if not 1 <= K <= MAX_TOP_K:
        raise ValueError(f"K must be in 1 .. {MAX_TOP_K}, got {K}")
    return (_per_row(ids, "ids", torch.int64, (T, K), dev), _per_row(teacher, "teacher", torch.float32, (T, K), dev), K)


def distill_topk_fwd(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, *,
                     V_true: Optional[int] = None, temperature: float = 1.0,
                     err_flag: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """rlk_distill_topk_fwd -> (loss, lse), fp32 [T] each: the KL divergence from the softmax of
    the teacher's top logits (fp32 [T, K], at columns ids int64 [T, K], -1: none) to
    softmax(logits / temperature), without a factor temperature^2, and the student's lse for the
    backward."""
    T, V, ld, code, dev = _rows(logits, "logits")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (logits, ids, teacher, err_flag)):
            return distill_topk_fwd(logits, ids, teacher, V_true=V_true, temperature=temperature, err_flag=err_flag)
    p = _teacher(ids, teacher, T, dev)
    V_true = _true_vocab(V_true, V)
    loss = torch.empty(T, dtype=torch.float32, device=logits.device)
    lse = torch.empty(T, dtype=torch.float32, device=logits.device)
    st = _load().rlk_distill_topk_fwd(logits.data_ptr(), code, T, ld, V_true, temperature, *p, loss.data_ptr(),
                                      lse.data_ptr(), _flag(err_flag, dev), _raw_stream(dev))
    if st:
        _check("rlk_distill_topk_fwd", st)
    return loss, lse


def distill_topk_bwd(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                     lse: torch.Tensor, g: torch.Tensor, *, V_true: Optional[int] = None,
                     temperature: float = 1.0, out: Optional[torch.Tensor] = None,
                     out_dtype: Optional[torch.dtype] = None,
                     err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rlk_distill_topk_bwd -> dlogits of sum_t g[t] loss[t], from the forward's lse. Shape, type
    and `out` as in :func:`token_logprobs_bwd`."""
    T, V, ld, code, dev = _rows(logits, "logits")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (logits, ids, teacher, lse, g, out, err_flag)):
            return distill_topk_bwd(logits, ids, teacher, lse, g, V_true=V_true, temperature=temperature, out=out,
                                    out_dtype=out_dtype, err_flag=err_flag)
    p = _teacher(ids, teacher, T, dev)
    lse_p = _per_row(lse, "lse", torch.float32, (T,), dev)
    g_p = _per_row(g, "g", torch.float32, (T,), dev)
    V_true = _true_vocab(V_true, V)
    dlogits, d = _gradient(logits, T, V, out, out_dtype)
    st = _load().rlk_distill_topk_bwd(logits.data_ptr(), code, T, ld, V_true, temperature, *p, lse_p, g_p, *d,
                                      _flag(err_flag, dev), _raw_stream(dev))
    if st:
        _check("rlk_distill_topk_bwd", st)
    if out is not None:
        _written((out,))
    return dlogits


def distill_topk_fwd_bwd(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                         g: torch.Tensor, *, V_true: Optional[int] = None, temperature: float = 1.0,
                         out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                         err_flag: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """rlk_distill_topk_fwd_bwd -> (loss, lse, dlogits): :func:`distill_topk_fwd` and
    :func:`distill_topk_bwd` in one call, for weights g known before the loss (a token mask over
    a count). The same bits; the logits are read once for rows of up to 53248 columns in 16-bit
    types and 13312 in float32, and for longer ones where they are few."""
    T, V, ld, code, dev = _rows(logits, "logits")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (logits, ids, teacher, g, out, err_flag)):
            return distill_topk_fwd_bwd(logits, ids, teacher, g, V_true=V_true, temperature=temperature, out=out,
                                        out_dtype=out_dtype, err_flag=err_flag)
    p = _teacher(ids, teacher, T, dev)
    g_p = _per_row(g, "g", torch.float32, (T,), dev)
    V_true = _true_vocab(V_true, V)
    loss, lse = torch.empty_like(g), torch.empty_like(g)
    dlogits, d = _gradient(logits, T, V, out, out_dtype)
    st = _load().rlk_distill_topk_fwd_bwd(logits.data_ptr(), code, T, ld, V_true, temperature, *p, g_p,
                                          loss.data_ptr(), lse.data_ptr(), *d, _flag(err_flag, dev),
                                          _raw_stream(dev))
    if st:
        _check("rlk_distill_topk_fwd_bwd", st)
    if out is not None:
        _written((out,))
    return loss, lse, dlogits


def bwd_dz_view(workspace: torch.Tensor, T: int, V_local: int) -> torch.Tensor:
    """The dz array at the start of a :func:`linear_logp_bwd` workspace as a bf16
    [T, round_up(V_local, 256)] tensor: a gradient written there (``out=``) is what the stages
    RLK_BWD_DH and RLK_BWD_DW turn into dH and dW."""
    Vd = -(-V_local // 256) * 256
    n = T * Vd * 2
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or workspace.numel() < n:
        raise ValueError(f"workspace must be a uint8 tensor of at least {n} bytes")
    return workspace[:n].view(torch.bfloat16).view(T, Vd)


class _OnceFn(torch.autograd.Function):
    """A gradient with a history that refuses: it depends on the logits and on the incoming gradients,
    and what has to differentiate it again must not take it for a constant. (once_differentiable
    looks at the incoming gradients alone, which are constants where the loss is linear in the output.)"""

    @staticmethod
    def forward(ctx, gradient, *inputs):
        return gradient.view_as(gradient)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("this operator is differentiable once: its gradient has no derivative")


def _once(gradient, *inputs):
    return _OnceFn.apply(gradient, *inputs) if torch.is_grad_enabled() else gradient   # enabled by create_graph alone


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, y, V_true, temperature):
        r = token_logprobs(logits, y, V_true=V_true, temperature=temperature)
        ctx.save_for_backward(logits, y, r.lse, r.entropy)
        ctx.args = dict(V_true=V_true, temperature=temperature)
        return r.logp, r.entropy

    @staticmethod
    def backward(ctx, g_logp, g_entropy):
        logits, y, lse, entropy = ctx.saved_tensors
        d = token_logprobs_bwd(logits, y, lse, entropy, g_logp.contiguous(), g_entropy.contiguous(), **ctx.args)
        return _once(d, logits, g_logp, g_entropy), None, None, None


def token_logprobs_autograd(logits: torch.Tensor, y: torch.Tensor, *, V_true: Optional[int] = None,
                            temperature: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """(logp, entropy) of each row, fp32 [T], differentiable in the logits (both gradients), once: a
    second derivative raises RuntimeError."""
    return _TokenLogprobsFn.apply(logits, y, V_true, temperature)


class _DistillTopkFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, V_true, temperature):
        loss, lse = distill_topk_fwd(logits, ids, teacher, V_true=V_true, temperature=temperature)
        ctx.save_for_backward(logits, ids, teacher, lse)
        ctx.args = dict(V_true=V_true, temperature=temperature)
        return loss

    @staticmethod
    def backward(ctx, g):
        logits, ids, teacher, lse = ctx.saved_tensors
        d = distill_topk_bwd(logits, ids, teacher, lse, g.contiguous(), **ctx.args)
        return _once(d, logits, g), None, None, None, None


def distill_topk(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, *,
                 V_true: Optional[int] = None, temperature: float = 1.0) -> torch.Tensor:
    """The distillation loss of each row, fp32 [T], differentiable in the logits (the teacher is
    a constant), once: a second derivative raises RuntimeError."""
    return _DistillTopkFn.apply(logits, ids, teacher, V_true, temperature)
