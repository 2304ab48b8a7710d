"""The trained layers beside the linear ones, and the scores of answers: embeddings, layer norms, log probabilities.

    y = dp.embedding(tokens, weight, scale=math.sqrt(D))             # tokens [B, T], weight [V, D]
    y = dp.layer_norm(x, weight, bias)                               # x [B, T, D]
    logprobs, entropy, top, indices = dp.token_logprobs(logits, tokens, top=20)

The three take part in autograd; embedding_backward, layer_norm_forward, layer_norm_backward,
token_logprobs_forward and token_logprobs_backward are the same computations without it.  dp.Embedding
and dp.LayerNorm are torch's modules over them, and what PrivacyEngine clips per example:
an embedding by the tokens and the output gradient, a layer norm by the per-example gradients, that its
backward pass leaves in place of the parameters' gradients.  embedding_desc and kept_desc describe both to ClipStep.

include/dpclip_seq.h states the formulas; the conventions are those of sequence.py (streams, checks, errors).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
import torch.autograd.forward_ad as _forward_ad
from torch.autograd.function import once_differentiable

from . import DP_BF16, DP_FP32, _check, _ptr, _stream
from . import sequence as _seq
from .sequence import _DTYPES, _INTS, _MOST, _call, _empty, _f32, _get, _keep, _no_tangents, _on, _opt, _rows_contiguous, _vector


class RowStrides(ctypes.Structure):
    """dp_row_strides: element strides of a [B, T, D] tensor."""
    _fields_ = [("b", ctypes.c_longlong), ("t", ctypes.c_longlong)]


class LogprobsDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "B", "T", "V", "K", "token_i64")] + \
               [("ld", ctypes.c_longlong), ("ld_grad", ctypes.c_longlong), ("tau", ctypes.c_float)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "w_dtype", "B", "T", "D", "has_bias", "per_example")] + \
               [("eps", ctypes.c_float), ("x", RowStrides), ("dy", RowStrides)]


class EmbeddingDesc(ctypes.Structure):
    """dp_embedding_desc; ClipStep takes it as a layer with the weight [V, D] and inputs (tokens, dY)."""
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "out_dtype", "B", "T", "V", "D", "index_i64", "padding")] + \
               [("scale", ctypes.c_float), ("ld", ctypes.c_longlong), ("dy", RowStrides)]
    has_bias = False

    @property
    def p(self) -> int:
        return self.V


class KeptDesc(ctypes.Structure):
    """A layer whose per-example gradients the caller has, fp32 [B, p D] or, with a bias, [B, p D + p];
    ClipStep's inputs for it are (gradients, None)."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "p", "D", "has_bias")]

    @property
    def n(self) -> int:
        return self.p * self.D + (self.p if self.has_bias else 0)


def embedding_desc(dtype: int, B: int, T: int, V: int, D: int, scale: float = 1.0, padding: Optional[int] = None,
                   index_i64: bool = False) -> EmbeddingDesc:
    """An embedding for ClipStep: tokens [B, T] (int32, or torch's int64 with index_i64) and the output gradient
    [B, T, D] of type dtype (DP_BF16 or DP_FP32), contiguous; the weight's gradient is fp32 [V, D]."""
    return EmbeddingDesc(dtype, DP_FP32, B, T, V, D, int(bool(index_i64)), -1 if padding is None else int(padding),
                         float(scale), D, RowStrides(T * D, D))


def kept_desc(B: int, p: int, D: int = 1, has_bias: bool = False) -> KeptDesc:
    """A layer of weight [p, D] for ClipStep whose per-example gradients the caller has (a layer norm: p its
    width, D = 1, the rows that layer_norm_backward(per_example=True) gives)."""
    if min(B, p, D) <= 0:
        raise ValueError(f"B={B}, p={p} and D={D} must be > 0")
    return KeptDesc(B, p, D, int(bool(has_bias)))


def _inputs_of(d):
    """(name, type, entries) of each input that a step is given for an EmbeddingDesc or a KeptDesc."""
    if isinstance(d, KeptDesc):
        return (("gradients", torch.float32, d.B * d.n),)
    rows = d.B * d.T
    own = d.dy.b == d.T * d.D and d.dy.t == d.D   # (other strides are the caller's: only the type is looked at)
    return (("tokens", torch.int64 if d.index_i64 else torch.int32, rows),
            ("output gradient", torch.bfloat16 if d.dtype == DP_BF16 else torch.float32, rows * d.D if own else 0))


def _check_inputs(wants, inputs) -> None:
    """Raises where a tensor (addresses are the caller's) is of another type or has not its entries one after another."""
    for (name, dtype, n), x in zip(wants, inputs):
        if isinstance(x, torch.Tensor) and (x.dtype != dtype or (n and (x.numel() < n or not x.is_contiguous()))):
            raise ValueError(f"{name}: contiguous {dtype} of {n} entries, got {x.dtype} {list(x.shape)}, strides {x.stride()}")


def _declare():
    v, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    P = ctypes.POINTER
    sig = {
        "dp_token_logprobs": (i, [P(LogprobsDesc)] + [v] * 8),
        "dp_token_logprobs_grad": (i, [P(LogprobsDesc)] + [v] * 8),
        "dp_layer_norm": (i, [P(LayerNormDesc)] + [v] * 7),
        "dp_layer_norm_grad_workspace": (sz, [P(LayerNormDesc)]),
        "dp_layer_norm_grad": (i, [P(LayerNormDesc)] + [v] * 8 + [sz, v]),
        "dp_example_sqnorms": (i, [v, i, sz, v, v]),
        "dp_example_sum": (i, [v, i, sz, v, v, i, v]),
        "dp_embedding": (i, [P(EmbeddingDesc)] + [v] * 4),
        "dp_embedding_order_size": (sz, [P(EmbeddingDesc)]),
        "dp_embedding_workspace": (sz, [P(EmbeddingDesc)]),
        "dp_embedding_order": (i, [P(EmbeddingDesc), v, v, v, sz, v]),
        "dp_embedding_sqnorms": (i, [P(EmbeddingDesc), v, v, v, v, sz, v]),
        "dp_embedding_grad": (i, [P(EmbeddingDesc), v, v, v, v, i, v, sz, v]),
        "dp_embedding_order_grad": (i, [P(EmbeddingDesc), v, v, v, v, v, i, v, sz, v]),
    }
    for name, (res, args) in sig.items():
        f = getattr(_seq._lib, name)
        f.restype, f.argtypes = res, args


_declare()


# ---- the C entry points ---------------------------------------------------------------
def _bytes(workspace, ws_bytes) -> int:
    if ws_bytes is not None:
        return ws_bytes
    return workspace.numel() * workspace.element_size() if workspace is not None else 0


def dp_token_logprobs(desc: LogprobsDesc, logits, tokens, logprobs, entropy, stats, top=None, top_indices=None,
                      stream=None) -> None:
    _check(_seq._lib.dp_token_logprobs(desc, _ptr(logits), _ptr(tokens), _ptr(logprobs), _ptr(entropy), _ptr(stats),
                                       _ptr(top), _ptr(top_indices), _stream(stream)))


def dp_token_logprobs_grad(desc: LogprobsDesc, logits, tokens, stats, entropy, d_logprobs, d_entropy, dlogits,
                           stream=None) -> None:
    _check(_seq._lib.dp_token_logprobs_grad(desc, _ptr(logits), _ptr(tokens), _ptr(stats), _ptr(entropy),
                                            _ptr(d_logprobs), _ptr(d_entropy), _ptr(dlogits), _stream(stream)))


def dp_layer_norm(desc: LayerNormDesc, X, W, b, Y, mean=None, rstd=None, stream=None) -> None:
    _check(_seq._lib.dp_layer_norm(desc, _ptr(X), _ptr(W), _ptr(b), _ptr(Y), _ptr(mean), _ptr(rstd), _stream(stream)))


def dp_layer_norm_grad_workspace(desc: LayerNormDesc) -> int:
    return int(_seq._lib.dp_layer_norm_grad_workspace(desc))


def dp_layer_norm_grad(desc: LayerNormDesc, dY, X, W, mean, rstd, dX, grads, workspace=None,
                       ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_seq._lib.dp_layer_norm_grad(desc, _ptr(dY), _ptr(X), _ptr(W), _ptr(mean), _ptr(rstd), _ptr(dX), _ptr(grads),
                                        _ptr(workspace), _bytes(workspace, ws_bytes), _stream(stream)))


def dp_example_sqnorms(grads, B: int, n: int, sqnorms, stream=None) -> None:
    _check(_seq._lib.dp_example_sqnorms(_ptr(grads), B, n, _ptr(sqnorms), _stream(stream)))


def dp_example_sum(grads, B: int, n: int, factors, out, accumulate: bool = False, stream=None) -> None:
    _check(_seq._lib.dp_example_sum(_ptr(grads), B, n, _ptr(factors), _ptr(out), int(bool(accumulate)), _stream(stream)))


def dp_embedding(desc: EmbeddingDesc, tokens, W, Y, stream=None) -> None:
    _check(_seq._lib.dp_embedding(desc, _ptr(tokens), _ptr(W), _ptr(Y), _stream(stream)))


def dp_embedding_order_size(desc: EmbeddingDesc) -> int:
    return int(_seq._lib.dp_embedding_order_size(desc))


def dp_embedding_workspace(desc: EmbeddingDesc) -> int:
    return int(_seq._lib.dp_embedding_workspace(desc))


def dp_embedding_order(desc: EmbeddingDesc, tokens, order, workspace, ws_bytes: Optional[int] = None,
                       stream=None) -> None:
    _check(_seq._lib.dp_embedding_order(desc, _ptr(tokens), _ptr(order), _ptr(workspace), _bytes(workspace, ws_bytes),
                                        _stream(stream)))


def dp_embedding_sqnorms(desc: EmbeddingDesc, order, dY, sqnorms, workspace, ws_bytes: Optional[int] = None,
                         stream=None) -> None:
    _check(_seq._lib.dp_embedding_sqnorms(desc, _ptr(order), _ptr(dY), _ptr(sqnorms), _ptr(workspace),
                                          _bytes(workspace, ws_bytes), _stream(stream)))


def dp_embedding_grad(desc: EmbeddingDesc, order, dY, factors, dW, workspace, ws_bytes: Optional[int] = None,
                      accumulate: bool = False, stream=None) -> None:
    _check(_seq._lib.dp_embedding_grad(desc, _ptr(order), _ptr(dY), _ptr(factors), _ptr(dW), int(bool(accumulate)),
                                       _ptr(workspace), _bytes(workspace, ws_bytes), _stream(stream)))


def dp_embedding_order_grad(desc: EmbeddingDesc, tokens, order, dY, factors, dW, workspace,
                            ws_bytes: Optional[int] = None, accumulate: bool = False, stream=None) -> None:
    _check(_seq._lib.dp_embedding_order_grad(desc, _ptr(tokens), _ptr(order), _ptr(dY), _ptr(factors), _ptr(dW),
                                             int(bool(accumulate)), _ptr(workspace), _bytes(workspace, ws_bytes),
                                             _stream(stream)))


_pass = torch._C._current_graph_task_id   # the backward pass that runs, or -1


# ---- argument checks ------------------------------------------------------------------
def _rows3(x, name: str):
    """x [B, ..., D] as [B, T, D]."""
    if x.dim() < 2 or not x.is_cuda or x.dtype not in _DTYPES:
        raise ValueError(f"{name}: a bf16 or fp32 CUDA tensor [B, ..., D], got {x.dtype} {tuple(x.shape)} on {x.device}")
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError(f"{name}: the innermost stride must be 1, got {x.stride()}")
    if max(x.shape) > _MOST:
        raise ValueError(f"{name}: sizes up to {_MOST}, got {tuple(x.shape)}")
    if x.dim() == 3:
        return x
    return x.unsqueeze(1) if x.dim() == 2 else x.flatten(1, -2)   # (a copy where no stride spans the middle)


# ---- layer norm -----------------------------------------------------------------------
def _norm_desc(x, weight, bias, eps, dy, mean, rstd, has_bias, per_example):
    _rows3(x, "x")
    B, T, D = x.shape
    if D == 0:
        raise ValueError("x: rows of at least one entry")
    for p, n in ((weight, "weight"), (bias, "bias")):
        _vector(p, x, (D,), tuple(_DTYPES), n)
    if bias is not None and (weight is None or bias.dtype != weight.dtype):
        raise ValueError("bias: comes with a weight of its type")
    if dy is not None:
        _rows3(dy, "dy")
        if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != x.device:
            raise ValueError(f"dy: {x.dtype} {tuple(x.shape)} on {x.device}, got {dy.dtype} {tuple(dy.shape)} on {dy.device}")
        _vector(mean, x, (B, T), (torch.float32,), "mean")
        _vector(rstd, x, (B, T), (torch.float32,), "rstd")
    d = LayerNormDesc(_DTYPES[x.dtype], DP_FP32 if weight is None else _DTYPES[weight.dtype], B, T, D, int(has_bias),
                      int(per_example), eps, RowStrides(*x.stride()[:2]),
                      RowStrides(*(dy.stride()[:2] if dy is not None else (0, 0))))
    if dy is not None and B * T:
        d.ws_bytes = dp_layer_norm_grad_workspace(d)
    return d


def _norm(x, weight, bias, eps, stats):
    if _forward_ad._current_level >= 0:
        _no_tangents(x, weight, bias)
    eps, shape = float(eps), x.shape
    if len(shape) != 3:
        x = _rows3(x, "x")
    dev, dtype = x.get_device(), x.dtype
    key = ("layer_norm", x.shape, x.stride(), dtype, dev, _opt(weight), _opt(bias), eps)
    d = _get(key) or _keep(key, _norm_desc(x, weight, bias, eps, None, None, None, False, False))
    device = x.device
    y = _empty(shape, dtype=dtype, device=device)
    mean = rstd = None
    if stats:
        mean, rstd = _empty(shape[:-1], dtype=_f32, device=device), _empty(shape[:-1], dtype=_f32, device=device)
    if d.B * d.T:
        _call(_seq._lib.dp_layer_norm, dev, d, x.data_ptr(), None if weight is None else weight.data_ptr(),
              None if bias is None else bias.data_ptr(), y.data_ptr(), None if mean is None else mean.data_ptr(),
              None if rstd is None else rstd.data_ptr())
    return y, mean, rstd


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """(y, mean, rstd): layer norm over the last dimension of x [B, ..., D], with each row's mean and
    1/sqrt(var + eps), fp32 [B, ...].  weight and bias: [D] of one type (bf16 or fp32), or None."""
    if stream is not None:
        with _on(stream, x.device):
            return _norm(x, weight, bias, eps, True)
    return _norm(x, weight, bias, eps, True)


def _statistics(s, shape, x, name):
    """Each row's statistic, of x's own `shape` but its last dimension (or in one dimension), as [B, T]."""
    n = x.shape[0] * x.shape[1]
    if (s.shape != shape[:-1] and s.shape != (n,)) or not s.is_contiguous():
        raise ValueError(f"{name}: contiguous {list(shape[:-1])}, got {list(s.shape)}")
    return s.view(x.shape[:2])


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True, per_example: bool = False, dx: bool = True,
                        params: bool = True, stream=None):
    """(dx, dw, db) for the gradient dy of layer_norm_forward's y; dw and db of the weight's type, db None
    without bias.  per_example: (dx, each), each fp32 [B, D] or with bias [B, 2 D], row i example i's own dw and
    then db.  dx=False or params=False: not formed (None)."""
    if stream is not None:
        with _on(stream, x.device):
            return layer_norm_backward(dy, x, weight, mean, rstd, bias, per_example, dx, params)
    if _forward_ad._current_level >= 0:
        _no_tangents(dy, x, weight, mean, rstd)
    bias, per_example, dx, params = bool(bias), bool(per_example), bool(dx), bool(params)
    shape = x.shape
    if len(shape) != 3:
        x = _rows3(x, "x")
        if dy.shape != shape and dy.shape != x.shape:
            raise ValueError(f"dy: {list(shape)} as x, got {list(dy.shape)}")
        dy = _rows3(dy, "dy")
    dev = x.get_device()
    if mean.dim() != 2:
        mean = _statistics(mean, shape, x, "mean")
    if rstd.dim() != 2:
        rstd = _statistics(rstd, shape, x, "rstd")
    key = ("layer_norm_backward", x.shape, x.stride(), x.dtype, dev, dy.shape, dy.stride(), dy.dtype, dy.get_device(),
           _opt(weight), _opt(mean), _opt(rstd), bias, per_example)
    d = _get(key) or _keep(key, _norm_desc(x, weight, None, 0.0, dy, mean, rstd, bias, per_example))
    device, D = x.device, d.D
    gx = _empty(shape, dtype=x.dtype, device=device) if dx else None
    grads = None
    if params and per_example:
        grads = _empty((d.B, 2 * D if bias else D), dtype=_f32, device=device)
    elif params:
        grads = _empty((2 if bias else 1, D), dtype=_f32 if weight is None else weight.dtype, device=device)
    if not d.B * d.T:
        if params:
            grads.zero_()
    elif dx or params:
        ws = _empty(d.ws_bytes, dtype=torch.uint8, device=device) if params and d.ws_bytes else None
        _call(_seq._lib.dp_layer_norm_grad, dev, d, dy.data_ptr(), x.data_ptr(), None if weight is None else weight.data_ptr(),
              mean.data_ptr(), rstd.data_ptr(), None if gx is None else gx.data_ptr(),
              None if grads is None else grads.data_ptr(), None if ws is None else ws.data_ptr(),
              0 if ws is None else d.ws_bytes)
    if per_example:
        return gx, grads
    if not params:
        return gx, None, None
    return gx, grads[0], grads[1] if bias else None   # (unbind costs the host three microseconds more)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, sink):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias, ctx.sink, ctx.within = bias is not None, sink, _pass()
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        want = ctx.needs_input_grad
        params = want[1] or want[2]
        dy = _rows_contiguous(dy)
        if ctx.sink is not None and params:   # each example's own, in place of their sum
            dx, each = layer_norm_backward(dy, x, weight, mean, rstd, ctx.has_bias, True, want[0])
            ctx.sink(ctx.within, each)
            return dx, None, None, None, None
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, ctx.has_bias, False, want[0], params)
        return dx, dw if want[1] else None, db if want[2] else None, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """layer_norm_forward's y, with its gradients."""
    return _layer_norm(x, weight, bias, eps, None, stream)


def _layer_norm(x, weight, bias, eps, sink, stream=None):
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad) or
                                    (bias is not None and bias.requires_grad)):
        if stream is not None:
            raise ValueError("a differentiable call runs on the current stream")
        return _LayerNorm.apply(x, weight, bias, float(eps), sink)
    if stream is not None:
        with _on(stream, x.device):
            return _norm(x, weight, bias, eps, False)[0]
    return _norm(x, weight, bias, eps, False)[0]


# ---- embedding ------------------------------------------------------------------------
def _tokens(tokens):
    if tokens.dim() < 1 or not tokens.is_cuda or tokens.dtype not in _INTS or not tokens.is_contiguous():
        raise ValueError(f"tokens: a contiguous int32 or int64 CUDA tensor [B, ...], got {tokens.dtype} {list(tokens.shape)} "
                         f"on {tokens.device}")
    if max(tokens.shape) > _MOST:
        raise ValueError(f"tokens: sizes up to {_MOST}, got {list(tokens.shape)}")


def _embedding_desc(tokens, weight, dy, V, scale, padding, factors, out_dtype):
    _tokens(tokens)
    B = tokens.shape[0]
    T = tokens.numel() // B if B else 0
    if weight is not None:
        if weight.dim() != 2 or weight.dtype not in _DTYPES or weight.device != tokens.device or weight.numel() == 0 or \
                max(weight.shape) > _MOST or (weight.stride(1) != 1 and weight.shape[1] > 1):
            raise ValueError(f"weight: bf16 or fp32 [V, D] with adjacent columns on {tokens.device}, got {weight.dtype} "
                             f"{list(weight.shape)} {weight.stride()} on {weight.device}")
        V, D = weight.shape
        dtype, ld, strides = weight.dtype, max(weight.stride(0), D) if V == 1 else weight.stride(0), (T * D, D)
    else:
        _rows3(dy, "dy")
        if dy.dim() != 3 or tuple(dy.shape[:2]) != (B, T) or dy.device != tokens.device or dy.shape[2] == 0:
            raise ValueError(f"dy {tuple(dy.shape)} on {dy.device} does not fit tokens {tuple(tokens.shape)} on {tokens.device}")
        D = dy.shape[2]
        dtype, ld, strides = dy.dtype, D, dy.stride()[:2]
        _vector(factors, tokens, (B,), (torch.float32,), "factors")
        if out_dtype not in _DTYPES:
            raise ValueError(f"dtype: bf16 or fp32, got {out_dtype}")
    if not 0 < V <= _MOST:
        raise ValueError(f"V={V} must be > 0 and up to {_MOST}")
    if padding is not None and not 0 <= padding < V:
        raise ValueError(f"padding={padding}: a token in [0, {V}), or None")
    d = EmbeddingDesc(_DTYPES[dtype], _DTYPES[out_dtype], B, T, V, D, int(tokens.dtype == torch.int64),
                      -1 if padding is None else padding, scale, ld, RowStrides(*strides))
    if B * T:
        d.order_bytes, d.ws_bytes = dp_embedding_order_size(d), dp_embedding_workspace(d)
    return d


def _lookup(tokens, weight, scale, padding):
    if _forward_ad._current_level >= 0:
        _no_tangents(weight)
    dev = tokens.get_device()
    key = ("embedding", tokens.shape, tokens.stride(), tokens.dtype, dev, weight.shape, weight.stride(), weight.dtype,
           weight.get_device(), scale, padding)
    d = _get(key) or _keep(key, _embedding_desc(tokens, weight, None, 0, scale, padding, None, torch.float32))
    y = _empty((*tokens.shape, d.D), dtype=weight.dtype, device=tokens.device)
    if d.B * d.T:
        _call(_seq._lib.dp_embedding, dev, d, tokens.data_ptr(), weight.data_ptr(), y.data_ptr())
    return y


def _grad_desc(tokens, dy, V, scale, padding, factors, dtype):
    """(dy as [B, T, D], descriptor) of a gradient call."""
    if _forward_ad._current_level >= 0:
        _no_tangents(dy, factors)
    V, scale = int(V), float(scale)
    if dy.dim() == tokens.dim() + 1 and dy.dim() != 3:
        if dy.shape[:-1] != tokens.shape:
            raise ValueError(f"dy {list(dy.shape)} does not fit tokens {list(tokens.shape)}")
        dy = _rows3(dy, "dy")
    key = ("embedding_backward", tokens.shape, tokens.stride(), tokens.dtype, tokens.get_device(), dy.shape, dy.stride(),
           dy.dtype, dy.get_device(), V, scale, padding, _opt(factors), dtype)
    return dy, _get(key) or _keep(key, _embedding_desc(tokens, None, dy, V, scale, padding, factors, dtype))


def _sorting(d, tokens):
    """Room for the tokens' order and a workspace as one array, and the addresses of the two."""
    both = _empty(d.order_bytes + d.ws_bytes, dtype=torch.uint8, device=tokens.device)
    order = both.data_ptr()
    return both, order, order + d.order_bytes   # (a multiple of 16)


def embedding_backward(tokens, dy, V: int, scale: float = 1.0, padding: Optional[int] = None, factors=None,
                       dtype=torch.float32, stream=None):
    """dW [V, D] of type dtype for the gradient dy [B, ..., D] of embedding's result: the sum over the
    examples, with factors (fp32 [B]) each example's part times its factor."""
    if stream is not None:
        with _on(stream, tokens.device):
            return embedding_backward(tokens, dy, V, scale, padding, factors, dtype)
    padding = None if padding is None else int(padding)
    dy, d = _grad_desc(tokens, dy, V, scale, padding, factors, dtype)
    dw = _empty((d.V, d.D), dtype=dtype, device=tokens.device)
    if not d.B * d.T:
        return dw.zero_()
    both, order, ws = _sorting(d, tokens)
    _call(_seq._lib.dp_embedding_order_grad, tokens.get_device(), d, tokens.data_ptr(), order, dy.data_ptr(),
          None if factors is None else factors.data_ptr(), dw.data_ptr(), 0, ws, d.ws_bytes)
    return dw


def embedding_sqnorms(tokens, dy, V: int, scale: float = 1.0, padding: Optional[int] = None, stream=None):
    """Each example's squared gradient norm fp32 [B]: of the gradient that it alone gives the weight."""
    if stream is not None:
        with _on(stream, tokens.device):
            return embedding_sqnorms(tokens, dy, V, scale, padding)
    padding = None if padding is None else int(padding)
    dy, d = _grad_desc(tokens, dy, V, scale, padding, None, torch.float32)
    sq = _empty(d.B, dtype=_f32, device=tokens.device)
    if not d.B * d.T:
        return sq.zero_()
    both, order, ws = _sorting(d, tokens)
    _call(_seq._lib.dp_embedding_order, tokens.get_device(), d, tokens.data_ptr(), order, ws, d.ws_bytes)
    _call(_seq._lib.dp_embedding_sqnorms, tokens.get_device(), d, order, dy.data_ptr(), sq.data_ptr(), ws, d.ws_bytes)
    return sq


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, padding, sinks):
        ctx.save_for_backward(tokens)
        ctx.opts, ctx.sinks, ctx.within = (weight.shape[0], scale, padding, weight.dtype), sinks, _pass()
        return _lookup(tokens, weight, scale, padding)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        tokens, = ctx.saved_tensors
        V, scale, padding, dtype = ctx.opts
        if ctx.sinks:   # what the examples' own gradients are formed from, in place of their sum
            for sink in ctx.sinks:
                sink(ctx.within, tokens, dy, scale, padding)
            return None, None, None, None, None
        return None, embedding_backward(tokens, _rows_contiguous(dy), V, scale, padding, dtype=dtype), None, None, None


def embedding(tokens, weight, scale: float = 1.0, padding: Optional[int] = None, stream=None):
    """scale * weight[tokens], [B, ..., D], with the gradient of weight [V, D]; tokens int32 or int64 [B, ...].
    The rows of the padding token have no gradient."""
    return _embedding(tokens, weight, scale, padding, (), stream)


def _embedding(tokens, weight, scale, padding, sinks, stream=None):
    scale, padding = float(scale), None if padding is None else int(padding)
    if torch.is_grad_enabled() and weight.requires_grad:
        if stream is not None:
            raise ValueError("a differentiable call runs on the current stream")
        return _Embedding.apply(tokens, weight, scale, padding, sinks)
    if stream is not None:
        with _on(stream, tokens.device):
            return _lookup(tokens, weight, scale, padding)
    return _lookup(tokens, weight, scale, padding)


# ---- log probabilities ----------------------------------------------------------------
def _logprobs_desc(logits, tokens, top, temperature, more):
    if logits.dim() != 3 or not logits.is_cuda or logits.dtype not in _DTYPES or logits.shape[2] == 0:
        raise ValueError(f"logits: a bf16 or fp32 CUDA tensor [B, T, V], got {logits.dtype} {tuple(logits.shape)} on "
                         f"{logits.device}")
    if max(logits.shape) > _MOST:
        raise ValueError(f"logits: sizes up to {_MOST}, got {tuple(logits.shape)}")
    B, T, V = logits.shape
    sb, sr, sv = logits.stride()
    if (sv != 1 and V > 1) or (B > 1 and T > 1 and sb != T * sr):
        raise ValueError(f"logits: rows at one stride and an innermost stride of 1, got strides {logits.stride()}")
    _vector(tokens, logits, (B, T), _INTS, "tokens")
    for x, shape, name in more:
        _vector(x, logits, (B, T) + shape, (torch.float32,), name)
    if not 0 <= top <= _MOST:
        raise ValueError(f"top={top}: from 0 to the kernel's 128")
    return LogprobsDesc(_DTYPES[logits.dtype], B, T, V, top, int(tokens is not None and tokens.dtype == torch.int64),
                        sr if T > 1 else sb if B > 1 else V, V, temperature)


def token_logprobs_forward(logits, tokens=None, top: int = 0, temperature: float = 1.0, stream=None):
    """(logprobs, entropy, stats, top_logprobs, top_indices) of logits [B, T, V] / temperature: the given
    tokens' log probabilities and each row's entropy, fp32 [B, T]; stats fp32 [B, T, 2] for
    token_logprobs_backward; and the `top` (at most 128) largest log probabilities fp32 [B, T, top] with their
    indices int32, largest first, of equal ones the lower index first (None with top=0).  tokens: int32 or
    int64 [B, T], negative where none is given (logprob 0); None: none at all."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs_forward(logits, tokens, top, temperature)
    if _forward_ad._current_level >= 0:
        _no_tangents(logits)
    top, temperature = int(top), float(temperature)
    dev = logits.get_device()
    key = ("token_logprobs", logits.shape, logits.stride(), logits.dtype, dev, _opt(tokens), top, temperature)
    d = _get(key) or _keep(key, _logprobs_desc(logits, tokens, top, temperature, ()))
    device, B, T = logits.device, d.B, d.T
    logprobs, entropy = _empty((B, T), dtype=_f32, device=device), _empty((B, T), dtype=_f32, device=device)
    stats = _empty((B, T, 2), dtype=_f32, device=device)
    best = _empty((B, T, top), dtype=_f32, device=device) if top else None
    indices = _empty((B, T, top), dtype=torch.int32, device=device) if top else None
    if B * T:
        _call(_seq._lib.dp_token_logprobs, dev, d, logits.data_ptr(), None if tokens is None else tokens.data_ptr(),
              logprobs.data_ptr(), entropy.data_ptr(), stats.data_ptr(), None if best is None else best.data_ptr(),
              None if indices is None else indices.data_ptr())
    return logprobs, entropy, stats, best, indices


def token_logprobs_backward(logits, tokens, stats, entropy, d_logprobs=None, d_entropy=None, temperature: float = 1.0,
                            stream=None):
    """The gradient of sum d_logprobs logprobs + d_entropy entropy (fp32 [B, T], None: 0) with respect to the
    logits; stats and entropy as token_logprobs_forward gave them."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs_backward(logits, tokens, stats, entropy, d_logprobs, d_entropy, temperature)
    if _forward_ad._current_level >= 0:
        _no_tangents(logits, stats, entropy, d_logprobs, d_entropy)
    temperature = float(temperature)
    dev = logits.get_device()
    key = ("token_logprobs_backward", logits.shape, logits.stride(), logits.dtype, dev, _opt(tokens), _opt(stats),
           _opt(entropy), _opt(d_logprobs), _opt(d_entropy), temperature)
    d = _get(key) or _keep(key, _logprobs_desc(logits, tokens, 0, temperature, (
        (stats, (2,), "stats"), (entropy, (), "entropy"), (d_logprobs, (), "d_logprobs"), (d_entropy, (), "d_entropy"))))
    grad = _empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if d.B * d.T:
        _call(_seq._lib.dp_token_logprobs_grad, dev, d, logits.data_ptr(), None if tokens is None else tokens.data_ptr(),
              stats.data_ptr(), entropy.data_ptr(), None if d_logprobs is None else d_logprobs.data_ptr(),
              None if d_entropy is None else d_entropy.data_ptr(), grad.data_ptr())
    return grad


class _Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, temperature):
        logprobs, entropy, stats, best, indices = token_logprobs_forward(logits, tokens, top, temperature)
        ctx.save_for_backward(logits, tokens, stats, entropy)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        if best is not None:
            ctx.mark_non_differentiable(best, indices)
        return logprobs, entropy, best, indices

    @staticmethod
    @once_differentiable
    def backward(ctx, dl, dh, *_):
        logits, tokens, stats, entropy = ctx.saved_tensors
        dl, dh = (None if g is None else g.contiguous() for g in (dl, dh))
        if dl is None and dh is None:
            return None, None, None, None
        return token_logprobs_backward(logits, tokens, stats, entropy, dl, dh, ctx.temperature), None, None, None


def token_logprobs(logits, tokens=None, top: int = 0, temperature: float = 1.0, stream=None):
    """(logprobs, entropy), with top > 0 (logprobs, entropy, top_logprobs, top_indices): see
    token_logprobs_forward.  logprobs and entropy carry gradients to the logits; top_logprobs and top_indices
    carry none (they are what distill_loss takes as `teacher` and `indices`)."""
    top, temperature = int(top), float(temperature)
    if torch.is_grad_enabled() and logits.requires_grad:
        if stream is not None:
            raise ValueError("a differentiable call runs on the current stream")
        logprobs, entropy, best, indices = _Logprobs.apply(logits, tokens, top, temperature)
    else:
        logprobs, entropy, _, best, indices = token_logprobs_forward(logits, tokens, top, temperature, stream)
    return (logprobs, entropy, best, indices) if top else (logprobs, entropy)


# ---- modules --------------------------------------------------------------------------
class LayerNorm(torch.nn.LayerNorm):
    """torch.nn.LayerNorm over the last dimension, by dp.layer_norm; PrivacyEngine clips its parameters.
    Inputs [B, ..., D], the examples first."""
    _sink = None   # where a backward pass leaves the per-example gradients (set by PrivacyEngine)

    def __init__(self, *args, **kwargs):
        super().__init__(*args, **kwargs)
        if len(self.normalized_shape) != 1:
            raise ValueError(f"normalized_shape {self.normalized_shape}: the last dimension only")

    def __getstate__(self):   # a copy is no engine's
        return {k: v for k, v in self.__dict__.items() if k != "_sink"}

    def forward(self, x):
        return _layer_norm(x, self.weight, self.bias, self.eps, self._sink)


class Embedding(torch.nn.Embedding):
    """torch.nn.Embedding by dp.embedding, times `scale`; PrivacyEngine clips its weight.  Tokens [B, ...],
    the examples first."""
    _sinks = ()   # where a backward pass leaves the tokens and the output gradient (set by PrivacyEngine)

    def __init__(self, *args, scale: float = 1.0, **kwargs):
        super().__init__(*args, **kwargs)
        if self.max_norm is not None or self.scale_grad_by_freq or self.sparse:
            raise ValueError("max_norm, scale_grad_by_freq and sparse gradients are not there")
        self.scale = float(scale)

    def __getstate__(self):   # a copy is no engine's
        return {k: v for k, v in self.__dict__.items() if k != "_sinks"}

    def forward(self, tokens):
        return _embedding(tokens.contiguous(), self.weight, self.scale, self.padding_idx, self._sinks)
