"""The sequence operators: rotary positions, attention and the distillation loss, with their gradients.

They run between the linear layers whose per-example gradients PrivacyEngine clips:

    table = dp.rotary_table(R=64, P=4096)                        # once
    q, k = dp.rotary(q, k, table)                                # q [B, T, Hq, D], k [B, T, Hk, D]
    o = dp.attention(q, k, v, causal=True, q_lens=lens, k_lens=lens)
    loss, rows = dp.distill_loss(logits, indices, teacher, labels=y, weights=w, temperature=2.0, alpha=0.1)
    loss.sum().backward(); engine.privatise(seed)

rotary, attention and distill_loss take part in autograd; attention_forward,
attention_backward and distill_loss_and_grad are the same computations without it.  The dp_*
functions marshal the arguments of the C entry points of include/dpclip_seq.h, which states
the formulas.  Work goes to the current stream of the tensors' device, or to `stream` as if it
were the current one: results and workspaces are allocated by torch for that stream, and the
usual rules for using a tensor on another stream apply.  An argument that does not fit raises ValueError (or
DPError, from the C side) before anything is launched.  Second and forward-mode derivatives are not there
and raise an error.  The kernels are launched past torch's dispatcher, so torch.jit.trace does not record them.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch
import torch.autograd.forward_ad as _forward_ad
from torch.autograd.function import once_differentiable

from . import DP_BF16, DP_FP32, _check, _lib, _ptr, _stream

DP_ROTARY_PLAIN, DP_ROTARY_LINEAR, DP_ROTARY_BASE, DP_ROTARY_PARTS = 0, 1, 2, 3
_SCALINGS = {"plain": DP_ROTARY_PLAIN, "linear": DP_ROTARY_LINEAR, "base": DP_ROTARY_BASE, "parts": DP_ROTARY_PARTS}


class Strides(ctypes.Structure):
    """dp_strides: element strides of a [B, T, H, D] tensor."""
    _fields_ = [("b", ctypes.c_longlong), ("t", ctypes.c_longlong), ("h", ctypes.c_longlong)]


class RotaryTableDesc(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int), ("R", ctypes.c_int), ("scaling", ctypes.c_int), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("context", ctypes.c_double), ("slow", ctypes.c_double),
                ("fast", ctypes.c_double)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "B", "T", "Hq", "Hk", "D", "R", "P", "interleaved", "inverse",
                                            "pos_i64")] + \
               [(n, Strides) for n in ("q", "k", "q_out", "k_out")]


class AttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "B", "T", "S", "Hq", "Hk", "D", "causal", "window")] + \
               [("scale", ctypes.c_float)] + \
               [(n, Strides) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")]


class DistillDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "teacher_dtype", "B", "T", "V", "K", "index_i64", "label_i64")] + \
               [("ld", ctypes.c_longlong), ("ld_grad", ctypes.c_longlong), ("tau", ctypes.c_float),
                ("alpha", ctypes.c_float)]


def _declare():
    v, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "dp_rotary_table": (ctypes.c_int, [P(RotaryTableDesc), v, v]),
        "dp_rotary": (ctypes.c_int, [P(RotaryDesc)] + [v] * 7),
        "dp_attention": (ctypes.c_int, [P(AttnDesc)] + [v] * 8),
        "dp_attention_grad_workspace": (sz, [P(AttnDesc)]),
        "dp_attention_grad": (ctypes.c_int, [P(AttnDesc)] + [v] * 12 + [sz, v]),
        "dp_distill": (ctypes.c_int, [P(DistillDesc)] + [v] * 10),
    }
    for name, (res, args) in sig.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = res, args


_declare()


# ---- the C entry points ---------------------------------------------------------------
def dp_rotary_table(desc: RotaryTableDesc, table, stream=None) -> None:
    _check(_lib.dp_rotary_table(desc, _ptr(table), _stream(stream)))


def dp_rotary(desc: RotaryDesc, Q, K, table, positions, Q_out, K_out, stream=None) -> None:
    _check(_lib.dp_rotary(desc, _ptr(Q), _ptr(K), _ptr(table), _ptr(positions), _ptr(Q_out), _ptr(K_out),
                          _stream(stream)))


def dp_attention(desc: AttnDesc, Q, K, V, O, lse=None, q_lens=None, k_lens=None, stream=None) -> None:
    _check(_lib.dp_attention(desc, _ptr(Q), _ptr(K), _ptr(V), _ptr(q_lens), _ptr(k_lens), _ptr(O), _ptr(lse),
                             _stream(stream)))


def dp_attention_grad_workspace(desc: AttnDesc) -> int:
    return int(_lib.dp_attention_grad_workspace(desc))


def dp_attention_grad(desc: AttnDesc, Q, K, V, O, lse, dO, dQ, dK, dV, workspace, q_lens=None, k_lens=None,
                      ws_bytes: Optional[int] = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.dp_attention_grad(desc, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), _ptr(dO), _ptr(q_lens),
                                  _ptr(k_lens), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace), ws_bytes,
                                  _stream(stream)))


def dp_distill(desc: DistillDesc, logits, indices, teacher, labels=None, weights=None, upstream=None, row_loss=None,
               loss=None, dlogits=None, stream=None) -> None:
    _check(_lib.dp_distill(desc, _ptr(logits), _ptr(indices), _ptr(teacher), _ptr(labels), _ptr(weights),
                           _ptr(upstream), _ptr(row_loss), _ptr(loss), _ptr(dlogits), _stream(stream)))


# ---- argument checks ------------------------------------------------------------------
_DTYPES = {torch.bfloat16: DP_BF16, torch.float32: DP_FP32}
_INTS = (torch.int32, torch.int64)
_MOST = 2 ** 31 - 1   # of a size: the descriptors' fields are C ints, which ctypes would fill modulo 2^32


def _heads(x, name: str) -> None:
    if x.dim() != 4 or not x.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor [B, T, H, D], got {tuple(x.shape)} on {x.device}")
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name}: bf16 or fp32, got {x.dtype}")
    if max(x.shape) > _MOST:
        raise ValueError(f"{name}: sizes up to {_MOST}, got {tuple(x.shape)}")
    if x.stride(3) != 1 and x.shape[3] > 1:
        raise ValueError(f"{name}: the innermost stride must be 1, got {x.stride()}")


def _like(x, ref, name: str) -> None:
    if x.dtype != ref.dtype or x.device != ref.device:
        raise ValueError(f"{name}: {x.dtype} on {x.device}, expected {ref.dtype} on {ref.device}")


def _vector(x, ref, shape, dtypes, name: str) -> None:
    """A contiguous device array of `shape`, or None."""
    if x is not None and (tuple(x.shape) != tuple(shape) or x.device != ref.device or not x.is_contiguous() or
                          x.dtype not in dtypes):
        raise ValueError(f"{name}: a contiguous {' or '.join(str(d) for d in dtypes)} tensor {list(shape)} on "
                         f"{ref.device}, got {x.dtype} {list(x.shape)} on {x.device}")


# Descriptors by what the checks and the descriptor look at of a call's tensors (shapes, strides,
# types and devices, never addresses or values) and by its options: a call like one that was
# checked before is neither checked nor described again.  The calls are a few microseconds of
# kernel at their smallest, so what is done per call is kept short.  Options are plain numbers
# before they are part of a key: one held in a tensor would be found by its identity, with the
# value that it had at an earlier call.
_descs: dict = {}
_get, _empty, _f32 = _descs.get, torch.empty, torch.float32
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _keep(key, d):
    if len(_descs) >= 1024:
        _descs.clear()
    _descs[key] = d
    return d


def _opt(x):
    """The key's part for an optional contiguous array."""
    return None if x is None else (x.shape, x.stride(), x.dtype, x.get_device())


def _no_tangents(*xs):
    """Forward-mode tangents would be dropped without a word: the kernels see addresses."""
    if any(x is not None and _forward_ad.unpack_dual(x).tangent is not None for x in xs):
        raise NotImplementedError("the sequence operators have no forward-mode derivatives")


def _on(stream, device):
    """`stream` (a torch stream or a handle) as the current one: what the call allocates then
    belongs to it, and a workspace that is dropped on return is not handed to another stream's
    work while the call still uses it."""
    if device.type != "cuda":
        return contextlib.nullcontext()   # refused by the checks
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    index = torch.cuda.current_device() if device.index is None else device.index
    if stream.device.index != index:
        raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{index}")
    return torch.cuda.stream(stream)


def _call(f, device, *args):
    """f(*args, stream) of the C side on the current stream of `device`, with that current."""
    stream = _current_stream(device)
    if device == _current_device():
        status = f(*args, stream)
    else:
        with torch.cuda.device(device):
            status = f(*args, stream)
    if status:
        _check(status)


# ---- rotary ---------------------------------------------------------------------------
def rotary_table(R: int, P: int, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                 context: float = 4096.0, slow: float = 1.0, fast: float = 32.0, device="cuda", stream=None):
    """Table fp32 [P, R] of the cosines and sines of R rotated entries at positions 0 .. P - 1.
    scaling: "plain", "linear" (positions / factor), "base" (theta stretched by factor) or
    "parts" (slow pairs interpolated, fast ones kept, by their turns over `context`)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling {scaling!r}: one of {sorted(_SCALINGS)}")
    if not (0 < P <= _MOST and 0 < R <= _MOST):
        raise ValueError(f"P={P} and R={R} must be > 0 and up to {_MOST}")
    device = torch.get_default_device() if device is None else torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"device: a CUDA device, got {device}")
    if stream is not None:
        with _on(stream, device):
            return rotary_table(R, P, theta, scaling, factor, context, slow, fast, device)
    table = torch.empty(P, R, dtype=torch.float32, device=device)
    _call(_lib.dp_rotary_table, table.get_device(),
          RotaryTableDesc(P, R, _SCALINGS[scaling], theta, factor, context, slow, fast), table.data_ptr())
    return table


def _rotary_desc(q, k, table, positions, interleaved, inverse):
    _heads(q, "q")
    B, T, Hq, D = q.shape
    if k is not None:
        _heads(k, "k")
        _like(k, q, "k")
        if k.shape[0] != B or k.shape[1] != T or k.shape[3] != D:
            raise ValueError(f"k {tuple(k.shape)} does not fit q {tuple(q.shape)}")
    if table.dim() != 2 or max(table.shape) > _MOST or table.dtype != torch.float32 or not table.is_contiguous() or table.device != q.device:
        raise ValueError("table: the contiguous fp32 [P, R] tensor of rotary_table, on q's device")
    _vector(positions, q, (B, T), _INTS, "positions")
    Hk = k.shape[2] if k is not None else 0
    return RotaryDesc(_DTYPES[q.dtype], B, T, Hq, Hk, D, table.shape[1], table.shape[0], int(interleaved),
                      int(inverse), int(positions is not None and positions.dtype == torch.int64),
                      Strides(*q.stride()[:3]), Strides(*(k.stride()[:3] if k is not None else (0, 0, 0))),
                      Strides(T * Hq * D, Hq * D, D), Strides(T * Hk * D, Hk * D, D))


def _rotary(q, k, table, positions, interleaved, inverse):
    if _forward_ad._current_level >= 0:
        _no_tangents(q, k, table)
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    key = (shape, q.stride(), dtype, dev, table.shape, table.stride(), table.dtype, table.get_device(), interleaved,
           inverse, None if k is None else (k.shape, k.stride(), k.dtype, k.get_device()),
           None if positions is None else (positions.shape, positions.stride(), positions.dtype, positions.get_device()))
    d = _get(key) or _keep(key, _rotary_desc(q, k, table, positions, interleaved, inverse))
    device = q.device
    qo = _empty(shape, dtype=dtype, device=device)
    ko = _empty(k.shape, dtype=dtype, device=device) if k is not None else None
    if d.B * d.T * (d.Hq + d.Hk) * d.D:
        _call(_lib.dp_rotary, dev, d, q.data_ptr(), None if k is None else k.data_ptr(), table.data_ptr(),
              None if positions is None else positions.data_ptr(), qo.data_ptr(), None if k is None else ko.data_ptr())
    return qo, ko


def _rows_contiguous(g):
    """A gradient as autograd hands it over (it may be expanded) with an innermost stride of 1."""
    return g if g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous()


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved, inverse):
        ctx.save_for_backward(table, positions)
        ctx.opts = (interleaved, inverse)
        return _rotary(q, k, table, positions, interleaved, inverse)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        table, positions = ctx.saved_tensors
        interleaved, inverse = ctx.opts
        dk = _rows_contiguous(dk) if dk is not None else None
        gq, gk = _rotary(_rows_contiguous(dq), dk, table, positions, interleaved, not inverse)
        return gq, gk, None, None, None, None


def rotary(q, k, table, positions=None, interleaved: bool = False, inverse: bool = False, stream=None):
    """(q', k') with the first table.shape[1] entries of every head turned by their position's
    angles; k may be None.  positions: int32 or int64 [B, T], None for 0 .. T - 1.  inverse
    turns the other way, the transposed rotation: the gradient, and what turns back unless the
    table has a magnitude ("parts", whose square then remains)."""
    interleaved, inverse = bool(interleaved), bool(inverse)
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if stream is not None:
            raise ValueError("a differentiable call runs on the current stream")
        return _Rotary.apply(q, k, table, positions, interleaved, inverse)
    if stream is not None:
        with _on(stream, q.device):
            return _rotary(q, k, table, positions, interleaved, inverse)
    return _rotary(q, k, table, positions, interleaved, inverse)


# ---- attention ------------------------------------------------------------------------
def _attn_desc(q, k, v, q_lens, k_lens, causal, window, scale, more=None):
    """Descriptor of a forward call, or with more = (o, lse, do) of a gradient call."""
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        _heads(x, n)
    _like(k, q, "k")
    _like(v, q, "v")
    B, T, Hq, D = q.shape
    S, Hk = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not fit q {tuple(q.shape)}")
    _vector(q_lens, q, (B,), (torch.int32,), "q_lens")
    _vector(k_lens, q, (B,), (torch.int32,), "k_lens")
    d = AttnDesc(_DTYPES[q.dtype], B, T, S, Hq, Hk, D, int(causal), window, scale or 0.0)
    if scale is not None and d.scale == 0:   # which the C side reads as the default
        raise ValueError(f"scale {scale}: 0 in fp32; None is 1/sqrt(D)")
    own, kv = Strides(T * Hq * D, Hq * D, D), Strides(S * Hk * D, Hk * D, D)   # of the results
    d.q, d.k, d.v, d.o = Strides(*q.stride()[:3]), Strides(*k.stride()[:3]), Strides(*v.stride()[:3]), own
    if more is not None:
        o, lse, do = more
        for x, n in ((o, "o"), (do, "do")):
            _heads(x, n)
            _like(x, q, n)
            if x.shape != q.shape:
                raise ValueError(f"{n} {tuple(x.shape)} is not shaped like q {tuple(q.shape)}")
        _vector(lse, q, (B, Hq, T), (torch.float32,), "lse")
        d.o, d.d_o, d.dq, d.dk, d.dv = Strides(*o.stride()[:3]), Strides(*do.stride()[:3]), own, kv, kv
        d.ws_bytes = dp_attention_grad_workspace(d)
    return d


def _options(causal, window, scale):
    # a window past a C int's range hides nothing, as the largest in it (below it: refused, as -1)
    return bool(causal), max(-1, min(int(window), _MOST)), None if scale is None else float(scale)


def attention_forward(q, k, v, causal: bool = False, window: int = 0, scale: Optional[float] = None, q_lens=None,
                      k_lens=None, stream=None):
    """(o, lse): attention of q [B, T, Hq, D] over k, v [B, S, Hk, D] and each query's log-sum-exp
    fp32 [B, Hq, T].  q_lens, k_lens: int32 [B], how many leading rows of each example are
    there; causal aligns the last query with the last key; window > 0 keeps the latest
    `window` keys.  scale: > 0, None for 1/sqrt(D).  A query that sees no key gives 0 and -inf."""
    if stream is not None:
        with _on(stream, q.device):
            return attention_forward(q, k, v, causal, window, scale, q_lens, k_lens)
    if _forward_ad._current_level >= 0:
        _no_tangents(q, k, v)
    causal, window, scale = _options(causal, window, scale)
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    key = (shape, q.stride(), dtype, dev, k.shape, k.stride(), k.dtype, k.get_device(), v.shape, v.stride(), v.dtype,
           v.get_device(), causal, window, scale, None if q_lens is None else _opt(q_lens),
           None if k_lens is None else _opt(k_lens))
    d = _get(key) or _keep(key, _attn_desc(q, k, v, q_lens, k_lens, causal, window, scale))
    device = q.device
    o = _empty(shape, dtype=dtype, device=device)
    lse = _empty((d.B, d.Hq, d.T), dtype=_f32, device=device)
    if not d.B * d.T * d.Hq * d.D * d.S * d.Hk:
        return o.zero_(), lse.fill_(-float("inf"))
    _call(_lib.dp_attention, dev, d, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          None if q_lens is None else q_lens.data_ptr(), None if k_lens is None else k_lens.data_ptr(), o.data_ptr(),
          lse.data_ptr())
    return o, lse


def attention_backward(q, k, v, o, lse, do, causal: bool = False, window: int = 0, scale: Optional[float] = None,
                       q_lens=None, k_lens=None, stream=None):
    """(dq, dk, dv) for the gradient `do` of attention_forward's o, the probabilities formed
    again from lse; the other arguments as in the forward call."""
    if stream is not None:
        with _on(stream, q.device):
            return attention_backward(q, k, v, o, lse, do, causal, window, scale, q_lens, k_lens)
    if _forward_ad._current_level >= 0:
        _no_tangents(q, k, v, o, lse, do)
    causal, window, scale = _options(causal, window, scale)
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    key = (shape, q.stride(), dtype, dev, k.shape, k.stride(), k.dtype, k.get_device(), v.shape, v.stride(), v.dtype,
           v.get_device(), causal, window, scale, None if q_lens is None else _opt(q_lens),
           None if k_lens is None else _opt(k_lens), o.shape, o.stride(), o.dtype, o.get_device(), lse.shape,
           lse.stride(), lse.dtype, lse.get_device(), do.shape, do.stride(), do.dtype, do.get_device())
    d = _get(key) or _keep(key, _attn_desc(q, k, v, q_lens, k_lens, causal, window, scale, (o, lse, do)))
    device = q.device
    dq = _empty(shape, dtype=dtype, device=device)
    dk = _empty(k.shape, dtype=dtype, device=device)
    dv = _empty(k.shape, dtype=dtype, device=device)
    if not d.B * d.T * d.Hq * d.D * d.S * d.Hk:
        return dq.zero_(), dk.zero_(), dv.zero_()
    ws = _empty(d.ws_bytes, dtype=torch.uint8, device=device)
    _call(_lib.dp_attention_grad, dev, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          do.data_ptr(), None if q_lens is None else q_lens.data_ptr(), None if k_lens is None else k_lens.data_ptr(),
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), d.ws_bytes)
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, window, scale, q_lens, k_lens):
        o, lse = attention_forward(q, k, v, causal, window, scale, q_lens, k_lens)
        ctx.save_for_backward(q, k, v, o, lse, q_lens, k_lens)
        ctx.opts = (causal, window, scale)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, q_lens, k_lens = ctx.saved_tensors
        return attention_backward(q, k, v, o, lse, _rows_contiguous(do), *ctx.opts, q_lens, k_lens) + (None,) * 5


def attention(q, k, v, causal: bool = False, window: int = 0, scale: Optional[float] = None, q_lens=None, k_lens=None):
    """attention_forward's o, with its gradient."""
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        return _Attention.apply(q, k, v, *_options(causal, window, scale), q_lens, k_lens)
    return attention_forward(q, k, v, causal, window, scale, q_lens, k_lens)[0]


# ---- distillation ---------------------------------------------------------------------
def _distill_desc(logits, indices, teacher, labels, weights, upstream, temperature, alpha):
    if logits.dim() != 3 or not logits.is_cuda or logits.dtype not in _DTYPES or logits.shape[2] == 0:
        raise ValueError(f"logits: a bf16 or fp32 CUDA tensor [B, T, V], got {logits.dtype} {tuple(logits.shape)} on "
                         f"{logits.device}")
    if max(logits.shape) > _MOST:
        raise ValueError(f"logits: sizes up to {_MOST}, got {tuple(logits.shape)}")
    B, T, V = logits.shape
    sb, sr, sv = logits.stride()
    if (sv != 1 and V > 1) or (B > 1 and T > 1 and sb != T * sr):
        raise ValueError(f"logits: rows at one stride and an innermost stride of 1, got strides {logits.stride()}")
    if indices.dim() != 3 or teacher.dtype not in _DTYPES:
        raise ValueError("indices and teacher: [B, T, K], teacher bf16 or fp32")
    K = indices.shape[2]
    _vector(indices, logits, (B, T, K), _INTS, "indices")
    _vector(teacher, logits, (B, T, K), tuple(_DTYPES), "teacher")
    _vector(labels, logits, (B, T), _INTS, "labels")
    _vector(weights, logits, (B, T), (torch.float32,), "weights")
    _vector(upstream, logits, (B,), (torch.float32,), "upstream")
    return DistillDesc(_DTYPES[logits.dtype], _DTYPES[teacher.dtype], B, T, V, min(K, _MOST), int(indices.dtype == torch.int64),
                       int(labels is not None and labels.dtype == torch.int64), sr if T > 1 else sb if B > 1 else V, V,
                       temperature, alpha)


def _distill(logits, indices, teacher, labels, weights, upstream, temperature, alpha, want_loss, want_grad, stream=None):
    if stream is not None:
        with _on(stream, logits.device):
            return _distill(logits, indices, teacher, labels, weights, upstream, temperature, alpha, want_loss, want_grad)
    if _forward_ad._current_level >= 0:
        _no_tangents(logits, teacher, weights, upstream)
    temperature, alpha = float(temperature), float(alpha)
    shape, dtype, dev = logits.shape, logits.dtype, logits.get_device()
    key = (shape, logits.stride(), dtype, dev, indices.shape, indices.stride(), indices.dtype, indices.get_device(),
           teacher.shape, teacher.stride(), teacher.dtype, teacher.get_device(), temperature, alpha, _opt(labels),
           _opt(weights), _opt(upstream))
    d = _get(key) or _keep(key, _distill_desc(logits, indices, teacher, labels, weights, upstream, temperature, alpha))
    device = logits.device
    loss = rows = grad = None
    if want_loss:
        loss = _empty(d.B, dtype=_f32, device=device)
        rows = _empty((d.B, d.T), dtype=_f32, device=device)
    if want_grad:
        grad = _empty(shape, dtype=dtype, device=device)
    if not d.B * d.T:
        return (loss.zero_() if want_loss else None), rows, grad
    _call(_lib.dp_distill, dev, d, logits.data_ptr(), indices.data_ptr(), teacher.data_ptr(),
          None if labels is None else labels.data_ptr(), None if weights is None else weights.data_ptr(),
          None if upstream is None else upstream.data_ptr(), None if rows is None else rows.data_ptr(),
          None if loss is None else loss.data_ptr(), None if grad is None else grad.data_ptr())
    return loss, rows, grad


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, indices, teacher, labels, weights, temperature, alpha):
        loss, rows, _ = _distill(logits, indices, teacher, labels, weights, None, temperature, alpha, True, False)
        ctx.save_for_backward(logits, indices, teacher, labels, weights)
        ctx.opts = (temperature, alpha)
        ctx.mark_non_differentiable(rows)
        return loss, rows

    @staticmethod
    @once_differentiable
    def backward(ctx, up, _):
        logits, indices, teacher, labels, weights = ctx.saved_tensors
        grad = _distill(logits, indices, teacher, labels, weights, up.float().contiguous(), *ctx.opts, False, True)[2]
        return grad, None, None, None, None, None, None


def distill_loss(logits, indices, teacher, labels=None, weights=None, temperature: float = 1.0, alpha: float = 0.0,
                 stream=None):
    """(loss, rows): each example's distillation loss fp32 [B] and its weighted tokens' losses
    fp32 [B, T].  logits [B, T, V] of the student; indices (int32 or int64, -1: no entry) and
    teacher [B, T, K] the teacher's top logits; labels [B, T] (negative: none); weights fp32
    [B, T].  loss carries the gradient with respect to the logits."""
    if torch.is_grad_enabled() and logits.requires_grad:
        if stream is not None:
            raise ValueError("a differentiable call runs on the current stream")
        return _Distill.apply(logits, indices, teacher, labels, weights, float(temperature), float(alpha))
    return _distill(logits, indices, teacher, labels, weights, None, temperature, alpha, True, False, stream)[:2]


def distill_loss_and_grad(logits, indices, teacher, labels=None, weights=None, upstream=None, temperature: float = 1.0,
                          alpha: float = 0.0, stream=None):
    """(loss, dlogits) in one pass over the logits: distill_loss and the gradient of
    sum_i upstream_i loss_i (upstream fp32 [B], None: 1), the G of the layer that made them."""
    loss, _, grad = _distill(logits, indices, teacher, labels, weights, upstream, temperature, alpha, True, True, stream)
    return loss, grad
