"""Operators around the head in a training step: embedding lookup (:func:`embedding_fwd`) and the
table's gradient (:func:`embedding_bwd`, new or added to the head's dW of a tied model), layer norm
and its gradient (:func:`layer_norm_fwd`, :func:`layer_norm_bwd`), and the norm over all gradients
(:func:`grad_norm`) with clipping (:func:`clip_grad_norm`). Where gradients are shards, that norm is the
shards' own.

Argument marshalling around the C entry points of the same names (include/rlk.h states their
mathematics, special rows and errors); all arithmetic runs in the library's CUDA kernels. Rows are
[T, H] CUDA tensors of bfloat16, float16 or float32 with contiguous rows (stride(1) == 1; stride(0) is
free). Work is enqueued on ``stream`` (default: the current stream of the tensors' device); with a
``stream`` given, outputs are allocated on it and the inputs are recorded as used there.

:func:`embedding` and :func:`layer_norm` are the autograd forms.
"""
from __future__ import annotations

import array
import functools
from operator import attrgetter
from typing import Optional, Sequence, Tuple, Union

import torch

from ._binding import _check, _load
from .logits import _DTYPES, RLK_DTYPE_F32, _away, _elsewhere, _flag, _once, _per_row, _raw_stream, _rows, _written

MAX_TENSORS = 1 << 14


def _result(like: torch.Tensor, rows: int, cols: int, out, out_dtype, name: str):
    """The tensor to fill -- `out` ([rows, cols], rows contiguous) or a new one -- with its address, dtype
    code and row distance."""
    if out is None:
        dtype = out_dtype or like.dtype
        code = _DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"out_dtype must be one of {[str(d) for d in _DTYPES]}, got {dtype}")
        r = torch.empty((rows, cols), dtype=dtype, device=like.device)
        return r, code, max(cols, 1)
    oT, oH, old, code, dev = _rows(out, name)
    if oT != rows or oH != cols:
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(out.shape)}")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"{name} must be {out_dtype}, got {out.dtype}")
    if dev != like.get_device():
        raise ValueError(f"{name} must be on {like.device}, got {out.device}")
    return out, code, old


def _tokens(ids, T, dev):
    """The address of the token ids; T None: however many there are."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if T is None and ids.dim() != 1:
        raise ValueError(f"ids must have 1 dim, got {tuple(ids.shape)}")
    return _per_row(ids, "ids", torch.int64, ids.shape if T is None else (T,), dev)


def _scratch(nbytes: int, like: torch.Tensor, workspace: Optional[torch.Tensor]):
    """A workspace of at least nbytes, its address and its size."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        return ws, ws.data_ptr(), nbytes
    if not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if workspace.get_device() != like.get_device():
        raise ValueError(f"workspace must be on {like.device}, got {workspace.device}")
    if workspace.numel() < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace, workspace.data_ptr(), workspace.numel()


# --------------------------------------------------------------------------- embedding


def embedding_fwd(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, V_true: Optional[int] = None,
                  vocab_start: int = 0, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, err_flag: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """rlk_embedding_fwd -> [T, H]: scale * table[ids - vocab_start], ids int64 [T]. The table is [V, H],
    or the shard of one that starts at token vocab_start; id -1 (padding) and tokens of other shards give zero
    rows. V_true (default: where the table ends) bounds the tokens. The result has the table's type (or
    out_dtype: bfloat16 for float32 tables); `out` supplies it."""
    V, H, ld, code, dev = _rows(table, "table")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (table, ids, out, err_flag)):
            return embedding_fwd(table, ids, scale=scale, V_true=V_true, vocab_start=vocab_start, out=out,
                                 out_dtype=out_dtype, err_flag=err_flag)
    p = _tokens(ids, None, dev)
    T = ids.shape[0]
    x, xcode, xld = _result(table, T, H, out, out_dtype, "out")
    st = _load().rlk_embedding_fwd(table.data_ptr(), code, V, H, ld, vocab_start,
                                   vocab_start + V if V_true is None else V_true, p, T, scale, x.data_ptr(), xcode, xld,
                                   _flag(err_flag, dev), _raw_stream(dev))
    if st:
        _check("rlk_embedding_fwd", st)
    if out is not None:
        _written((out,))
    return x


@functools.lru_cache(maxsize=256)   # they follow from the sizes alone, and a small call is bound by the host
def embedding_bwd_workspace_bytes(T: int, H: int) -> int:
    return int(_load().rlk_embedding_bwd_workspace(T, H))


def embedding_bwd(dout: torch.Tensor, ids: torch.Tensor, V: int, *, scale: float = 1.0, V_true: Optional[int] = None,
                  vocab_start: int = 0, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                  err_flag: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """rlk_embedding_bwd -> dW, fp32 [V, H]: the gradient of the V rows of the table (or shard) that
    :func:`embedding_fwd` read, from dout [T, H]. `out` supplies dW; accumulate adds to what it holds (the dW of
    :func:`linear_logp_bwd`, where table and head are one weight) and leaves the rows of other tokens alone."""
    T, H, ld, code, dev = _rows(dout, "dout")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (dout, ids, out, err_flag, workspace)):
            return embedding_bwd(dout, ids, V, scale=scale, V_true=V_true, vocab_start=vocab_start, out=out,
                                 accumulate=accumulate, err_flag=err_flag, workspace=workspace)
    p = _tokens(ids, T, dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out, the gradient to add to")
    if out is None:
        dW = torch.empty((V, H), dtype=torch.float32, device=dout.device)
        at = dW.data_ptr()
    else:
        dW = out
        at = _per_row(out, "out", torch.float32, (V, H), dev)
    ws, wp, nbytes = _scratch(embedding_bwd_workspace_bytes(T, H), dout, workspace)
    st = _load().rlk_embedding_bwd(dout.data_ptr(), code, T, H, ld, p, V, vocab_start,
                                   vocab_start + V if V_true is None else V_true, scale, at, accumulate,
                                   _flag(err_flag, dev), wp, nbytes, _raw_stream(dev))
    if st:
        _check("rlk_embedding_bwd", st)
    if out is not None:
        _written((out,))
    return dW


# --------------------------------------------------------------------------- layer norm


def _vectors(weight, bias, x, H, dev):
    """Addresses of weight and bias and their common dtype code."""
    p, code = [], None
    for v, name in ((weight, "weight"), (bias, "bias")):
        if v is None:
            p.append(None)
            continue
        if not isinstance(v, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        c = _DTYPES.get(v.dtype)
        if c is None or (v.dtype != x.dtype and v.dtype is not torch.float32) or (code is not None and c != code):
            raise TypeError(f"weight and bias must both be {x.dtype} or both torch.float32, got {v.dtype}")
        code = c
        p.append(_per_row(v, name, v.dtype, (H,), dev))
    return p[0], p[1], RLK_DTYPE_F32 if code is None else code


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-5, centered: bool = True, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, err_flag: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """rlk_layer_norm_fwd -> (y, mean, rstd): (x - mean) rstd weight + bias of each row of x [T, H], mean and
    rstd fp32 [T] for the backward. centered=False takes the mean as 0 (the root-mean-square norm; mean is then
    None). weight and bias [H] are of x's type or float32. y has x's type (or out_dtype: bfloat16 for float32
    rows); `out` supplies it, x itself included."""
    T, H, ld, code, dev = _rows(x, "x")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (x, weight, bias, out, err_flag)):
            return layer_norm_fwd(x, weight, bias, eps=eps, centered=centered, out=out, out_dtype=out_dtype,
                                  err_flag=err_flag)
    w, b, wcode = _vectors(weight, bias, x, H, dev)
    y, ycode, yld = _result(x, T, H, out, out_dtype, "out")
    mean = torch.empty(T, dtype=torch.float32, device=x.device) if centered else None
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    st = _load().rlk_layer_norm_fwd(x.data_ptr(), code, T, H, ld, w, b, wcode, centered, eps, y.data_ptr(), ycode, yld,
                                    mean.data_ptr() if centered else None, rstd.data_ptr(), _flag(err_flag, dev),
                                    _raw_stream(dev))
    if st:
        _check("rlk_layer_norm_fwd", st)
    if out is not None:
        _written((out,))
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def layer_norm_bwd_workspace_bytes(T: int, H: int) -> int:
    return int(_load().rlk_layer_norm_bwd_workspace(T, H))


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: Optional[torch.Tensor],
                   rstd: torch.Tensor, *, want_dx: bool = True, want_dw: bool = True, want_db: bool = True,
                   out: Optional[torch.Tensor] = None, err_flag: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """rlk_layer_norm_bwd -> (dx, dw, db): the gradients of :func:`layer_norm_fwd` from dy [T, H] and the forward's
    mean (None: not centered) and rstd; dx in x's type, dw and db fp32 [H], None for those not wanted. `out`
    supplies dx, dy or x themselves included (of x's type)."""
    T, H, ld, code, dev = _rows(x, "x")
    if _away(stream, dev):
        with _elsewhere(stream, dev, (dy, x, weight, mean, rstd, out, err_flag, workspace)):
            return layer_norm_bwd(dy, x, weight, mean, rstd, want_dx=want_dx, want_dw=want_dw, want_db=want_db, out=out,
                                  err_flag=err_flag, workspace=workspace)
    dT, dH, dld, dcode, ddev = _rows(dy, "dy")
    if dT != T or dH != H:
        raise ValueError(f"dy must have shape {(T, H)}, got {tuple(dy.shape)}")
    if ddev != dev:
        raise ValueError(f"dy must be on {x.device}, got {dy.device}")
    if not (want_dx or want_dw or want_db):
        raise ValueError("nothing is wanted of the backward")
    w, _, wcode = _vectors(weight, None, x, H, dev)
    m = None if mean is None else _per_row(mean, "mean", torch.float32, (T,), dev)
    r = _per_row(rstd, "rstd", torch.float32, (T,), dev)
    dx, xp, xld = None, None, H
    if want_dx:
        dx, _, xld = _result(x, T, H, out, x.dtype, "out")
        xp = dx.data_ptr()
    elif out is not None:
        raise ValueError("out is dx, which is not wanted")
    dw = torch.empty(H, dtype=torch.float32, device=x.device) if want_dw else None
    db = torch.empty(H, dtype=torch.float32, device=x.device) if want_db else None
    ws, wp, nbytes = _scratch(layer_norm_bwd_workspace_bytes(T, H), x, workspace)
    st = _load().rlk_layer_norm_bwd(dy.data_ptr(), dcode, dld, x.data_ptr(), code, ld, T, H, w, wcode, m, r, xp, xld,
                                    dw.data_ptr() if want_dw else None, db.data_ptr() if want_db else None,
                                    _flag(err_flag, dev), wp, nbytes, _raw_stream(dev))
    if st:
        _check("rlk_layer_norm_bwd", st)
    if out is not None:
        _written((out,))
    return dx, dw, db


# --------------------------------------------------------------------------- all gradients


# Properties of many tensors without a line of Python for each: 216 gradients take 50 us, with a loop 100.
_data_ptr, _numel, _device_of = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device
_contiguous, _dtype_of = torch.Tensor.is_contiguous, attrgetter("dtype")


def _listed(tensors, name: str, dev: int):
    """Addresses and dtype codes of dense CUDA tensors of one device, as arrays."""
    if not tensors or set(map(_device_of, tensors)) != {dev}:
        raise ValueError(f"{name} must all be CUDA tensors of one device")
    if not all(map(_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    dtypes = list(map(_dtype_of, tensors))
    for d in set(dtypes):
        if d not in _DTYPES:
            raise TypeError(f"{name} must be of {[str(d) for d in _DTYPES]}, got {d}")
    if dtypes.count(dtypes[0]) == len(dtypes):
        codes = array.array("i", [_DTYPES[dtypes[0]]]) * len(dtypes)
    else:
        codes = array.array("i", map(_DTYPES.__getitem__, dtypes))
    return array.array("Q", map(_data_ptr, tensors)), codes


def _address(a: array.array) -> int:
    return a.buffer_info()[0]


def _gradients(grads):
    grads = (grads,) if isinstance(grads, torch.Tensor) else tuple(grads)
    if not grads:
        raise ValueError("there must be a gradient at least")
    if len(grads) > MAX_TENSORS:
        raise ValueError(f"at most {MAX_TENSORS} gradients, got {len(grads)}")
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError("gradients must be torch.Tensors")
    dev = grads[0].get_device()
    if dev < 0:
        raise ValueError("gradients must be CUDA tensors")
    return grads, dev


@functools.lru_cache(maxsize=256)
def grad_norm_workspace_bytes(n: int) -> int:
    """Of :func:`grad_norm` and :func:`clip_grad_norm` over n tensors."""
    return int(_load().rlk_grad_norm_workspace(n))


def _norm_result(out, like, dev):
    if out is None:
        return torch.empty((), dtype=torch.float32, device=like.device)
    _per_row(out, "norm", torch.float32, (), dev)
    return out


def grad_norm(grads: Union[torch.Tensor, Sequence[torch.Tensor]], *, norm: Optional[torch.Tensor] = None,
              err_flag: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """rlk_grad_norm -> the 2-norm over all elements of the gradients (contiguous CUDA tensors of any shapes), an
    fp32 tensor without dimensions; `norm` supplies it."""
    grads, dev = _gradients(grads)
    if _away(stream, dev):
        with _elsewhere(stream, dev, (*grads, norm, err_flag, workspace)):
            return grad_norm(grads, norm=norm, err_flag=err_flag, workspace=workspace)
    at, codes = _listed(grads, "gradients", dev)
    sizes = array.array("q", map(_numel, grads))
    n = len(grads)
    r = _norm_result(norm, grads[0], dev)
    ws, wp, nbytes = _scratch(grad_norm_workspace_bytes(n), grads[0], workspace)
    st = _load().rlk_grad_norm(_address(at), _address(sizes), _address(codes), n, r.data_ptr(), _flag(err_flag, dev),
                               wp, nbytes, _raw_stream(dev))
    if st:
        _check("rlk_grad_norm", st)
    if norm is not None:
        _written((norm,))
    return r


def clip_grad_norm(grads: Union[torch.Tensor, Sequence[torch.Tensor]], max_norm: float, *,
                   out: Optional[Union[torch.Tensor, Sequence[torch.Tensor]]] = None,
                   norm: Optional[torch.Tensor] = None, err_flag: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rlk_clip_grad_norm -> the norm over all gradients, as :func:`grad_norm`, and the gradients times max_norm / norm
    where that is below 1: in place, or into `out`, tensors of the same element counts (and types, or bfloat16 for
    float32). A norm that is not finite leaves them unscaled and raises RLK_FLAG_NONFINITE in err_flag."""
    grads, dev = _gradients(grads)
    outs = grads if out is None else ((out,) if isinstance(out, torch.Tensor) else tuple(out))
    if _away(stream, dev):
        with _elsewhere(stream, dev, (*grads, *(() if out is None else outs), norm, err_flag, workspace)):
            return clip_grad_norm(grads, max_norm, out=None if out is None else outs, norm=norm, err_flag=err_flag,
                                  workspace=workspace)
    if not max_norm > 0:   # NaN neither
        raise ValueError(f"max_norm must be above 0, got {max_norm}")
    at, codes = _listed(grads, "gradients", dev)
    to, ocodes = at, codes
    if out is not None:
        to, ocodes = _listed(outs, "out", dev)
    sizes = array.array("q", map(_numel, grads))
    if out is not None and array.array("q", map(_numel, outs)) != sizes:
        raise ValueError("out must hold a tensor of each gradient's element count")
    n = len(grads)
    r = _norm_result(norm, grads[0], dev)
    ws, wp, nbytes = _scratch(grad_norm_workspace_bytes(n), grads[0], workspace)
    st = _load().rlk_clip_grad_norm(_address(at), _address(sizes), _address(codes), n, max_norm, _address(to),
                                    _address(ocodes), r.data_ptr(), _flag(err_flag, dev), wp, nbytes,
                                    _raw_stream(dev))
    if st:
        _check("rlk_clip_grad_norm", st)
    _written(outs if norm is None else (*outs, norm))
    return r


# --------------------------------------------------------------------------- autograd


def _dense(g: torch.Tensor) -> torch.Tensor:
    """An incoming gradient as the entry points take rows (an expanded one has none of its own)."""
    return g if g.stride(1) == 1 and g.stride(0) >= g.shape[1] else g.contiguous()


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale, V_true, out_dtype):
        ctx.save_for_backward(ids)
        ctx.args = dict(scale=scale, V_true=V_true)
        ctx.V = table.shape[0]
        return embedding_fwd(table, ids, scale=scale, V_true=V_true, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, g):
        ids, = ctx.saved_tensors
        return _once(embedding_bwd(_dense(g), ids, ctx.V, **ctx.args), g), None, None, None, None


def embedding(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, V_true: Optional[int] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """:func:`embedding_fwd`, differentiable in the table, once: a second derivative raises RuntimeError. The
    gradient is dense: computed in fp32, then cast to the table's type by autograd, as that of
    :func:`linear_logp`'s W."""
    return _EmbeddingFn.apply(table, ids, scale, V_true, out_dtype)


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, centered, out_dtype):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps=eps, centered=centered, out_dtype=out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, g):
        x, weight, mean, rstd = ctx.saved_tensors
        want_dx, want_dw, want_db = ctx.needs_input_grad[:3]
        dx, dw, db = layer_norm_bwd(_dense(g), x, weight, mean, rstd, want_dx=want_dx,
                                    want_dw=want_dw, want_db=want_db)
        again = [None if d is None else _once(d, g, x, *(() if weight is None else (weight,))) for d in (dx, dw, db)]
        return (*again, None, None, None)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, centered: bool = True, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """:func:`layer_norm_fwd`'s y, differentiable in x, weight and bias, once: a second derivative raises
    RuntimeError."""
    return _LayerNormFn.apply(x, weight, bias, eps, centered, out_dtype)
