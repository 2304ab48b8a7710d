"""Privatised gradients for a PyTorch model: A and G captured by autograd hooks.

The pages' privacy engine ([MixGhost] Appendix E; [FastClip] section 2) wraps a model so
that per-example clipping needs a few lines of code: the layer inputs A and the output
gradients G are taken from the ordinary forward and backward passes, the per-example
norms are formed from them (ghost norm or instantiation, [MixGhost] section 4), and the
clipped sum replaces the second back-propagation of the reweighted loss ([MixGhost] section
3.2) with one contraction per layer in this library.

Use (with a summed loss G_i is example i's own gradient; loss_reduction="mean" undoes the
1/B of an averaged loss):

    engine = PrivacyEngine(model, C=1.0, sigma=1.0)
    loss = criterion(model(x), y)          # reduction="sum"
    loss.backward()
    engine.privatise(seed)                 # param.grad <- (sum_i c_i g_i + sigma C z) / B
    optimizer.step()

Layers: nn.Linear (inputs [B, ..., d]; the middle dimensions are the rows T), nn.Conv1d,
nn.Conv2d and nn.Conv3d (square or cubic kernels, equal stride / padding / dilation in every
dimension), the conv layers with groups 1 and zero padding.  Conv2d/Conv3d layers whose input
arrives in PyTorch's channels_last memory format are handed over channels last (no layout
copy); their output gradients are brought to the same format.  dp.Embedding (tokens [B, ...]) is
clipped by the tokens and the output gradient, dp.LayerNorm (inputs [B, ..., D]) by the per-example gradients,
that its backward pass leaves in place of its parameters' gradients (their .grad is privatise's alone); torch's
own two modules are not taken.  A layer is called
once in a step, and its weight and bias are its own (of an embedding's or a layer norm's, a use outside the
layer is an error in the backward pass).  Every trainable parameter of the model must belong to such a layer.
A and G are those of the call that the backward pass reaches; calls that none reaches change nothing.
"""
from __future__ import annotations

from typing import List, Optional

from . import DP_BF16, DP_CONV1D, DP_CONV2D, DP_CONV3D, DP_FP32, DP_LINEAR, DP_NCHW, DP_NHWC, DP_NORM_AUTO, layer_desc
from .layers import Embedding, LayerNorm, embedding_desc, kept_desc
from .step import ClipStep


class PrivacyEngine:
    def __init__(self, model, C=1.0, sigma: float = 1.0, per_layer: bool = False, norm_mode: int = DP_NORM_AUTO,
                 keep_grads="auto", loss_reduction: str = "sum"):
        """loss_reduction: "sum" (G_i as captured) or "mean" (the captured output gradients
        carry a 1/B factor, undone before the norms)."""
        import torch.nn as nn
        convs = (nn.Conv1d, nn.Conv2d, nn.Conv3d)
        if loss_reduction not in ("sum", "mean"):
            raise ValueError("loss_reduction is 'sum' or 'mean'")
        self.loss_reduction = loss_reduction
        self.model = model
        self.C, self.sigma, self.per_layer = C, float(sigma), bool(per_layer)
        self.norm_mode, self.keep_grads = norm_mode, keep_grads
        self.layers: List = []
        owned = set()
        for m in model.modules():
            if isinstance(m, (nn.Linear, Embedding, LayerNorm) + convs) and m.weight is not None and m.weight.requires_grad:
                if isinstance(m, convs):
                    self._check_conv(m)
                bias = getattr(m, "bias", None)
                if bias is not None and not bias.requires_grad:
                    raise ValueError(f"{m}: a bias must be trainable with its weight")
                for what, prm in (("weight", m.weight), ("bias", bias)):
                    if prm is not None and id(prm) in owned:   # its gradient would be the last layer's part alone
                        raise ValueError(f"{m}: shares its {what} with another layer, which is not clipped here")
                    owned.add(id(prm))
                self.layers.append(m)
        for name, prm in model.named_parameters():
            if prm.requires_grad and id(prm) not in owned:
                raise ValueError(f"parameter {name}: only nn.Linear, nn.Conv1d/2d/3d, dp.Embedding and dp.LayerNorm "
                                 "layers have per-example clipping here; freeze it or leave it out of the model")
        if not self.layers:
            raise ValueError("the model has no trainable layer that is clipped here")
        self._acts: List = [None] * len(self.layers)
        self._grads: List = [None] * len(self.layers)
        self._options: List = [()] * len(self.layers)
        self._tasks = [-1] * len(self.layers)   # the backward pass that last reached each
        self._handles = []
        for m in self.layers:
            if isinstance(m, LayerNorm) and m._sink is not None:
                raise ValueError(f"{m}: another engine's (its detach() frees it)")
        self._sinks = []
        for i, m in enumerate(self.layers):
            if isinstance(m, (Embedding, LayerNorm)):   # their own backward passes give their parameters no gradient
                for prm in (m.weight, getattr(m, "bias", None)):
                    if prm is not None:
                        self._handles.append(prm.register_hook(self._elsewhere(m)))
            if isinstance(m, LayerNorm):
                m._sink = self._sink(i)
                continue
            if isinstance(m, Embedding):
                self._sinks.append(self._sink(i))
                m._sinks += (self._sinks[-1],)
                continue
            self._handles.append(m.register_forward_hook(self._fwd_hook(i)))
        self._step: Optional[ClipStep] = None
        self._key = None

    @staticmethod
    def _check_conv(m) -> None:
        k, s, p, d = m.kernel_size, m.stride, m.padding, m.dilation
        if isinstance(p, str) or m.groups != 1 or m.padding_mode != "zeros":
            raise ValueError(f"{m}: groups=1 and zero padding given as numbers only")
        if any(len(set(v)) != 1 for v in (k, s, p, d)):
            raise ValueError(f"{m}: square or cubic kernels with equal stride/padding/dilation in every dimension only")

    def _fwd_hook(self, i):
        import torch

        def hook(module, inputs, output):
            if module is not self.layers[i] or not output.requires_grad:
                return   # (a copy's call, or one that no backward pass reaches)
            a, within = inputs[0].detach(), torch._C._current_graph_task_id()

            def taken(g):                  # the gradient of the loss w.r.t. this call's output
                self._once(i, within)
                self._acts[i], self._grads[i] = a, g.detach()
            output.register_hook(taken)
        return hook

    def _sink(self, i):
        # of a layer norm: the per-example gradients; of an embedding: the tokens, the output gradient, and the
        # scale and padding token that the call had
        def sink(within, a, g=None, *options):
            self._once(i, within)
            self._acts[i], self._grads[i], self._options[i] = a, g, options
        return sink

    @staticmethod
    def _elsewhere(m):
        def hook(grad):   # None from the layer itself; what reaches it all the same, privatise would write over
            if grad is not None:
                raise RuntimeError(f"{m}: a parameter is used beside the layer's own call, which is not clipped here")
        return hook

    def _once(self, i, within: int) -> None:
        """Raises where one backward pass reaches layer i again: the first call's gradient would be lost.  within:
        the pass in which the call itself ran, -1 for none (a checkpointed segment is run again in the pass that
        differentiates it, and differentiated by one of its own)."""
        import torch
        task = within if within != -1 else torch._C._current_graph_task_id()
        if task == self._tasks[i]:
            raise RuntimeError(f"{self.layers[i]}: called more than once in a step, which is not clipped here")
        self._tasks[i] = task

    def detach(self) -> None:
        """Remove the hooks."""
        for h in self._handles:
            h.remove()
        self._handles = []
        for m in self.layers:
            if isinstance(m, LayerNorm):
                m._sink = None
            elif isinstance(m, Embedding):
                m._sinks = tuple(s for s in m._sinks if s not in self._sinks)
        self._sinks = []

    @staticmethod
    def _layout(m, a) -> int:
        import torch
        import torch.nn as nn
        if isinstance(m, nn.Conv2d) and a.dim() == 4 and not a.is_contiguous() and \
                a.is_contiguous(memory_format=torch.channels_last):
            return DP_NHWC
        if isinstance(m, nn.Conv3d) and a.dim() == 5 and not a.is_contiguous() and \
                a.is_contiguous(memory_format=torch.channels_last_3d):
            return DP_NHWC
        return DP_NCHW

    @staticmethod
    def _as_layout(x, layout: int, dtype):
        import torch
        x = x.to(dtype)
        if layout == DP_NHWC:
            return x.contiguous(memory_format=torch.channels_last if x.dim() == 4 else torch.channels_last_3d)
        return x.contiguous()

    def _descs(self, B: int, dtype: int, layouts):
        import torch
        import torch.nn as nn
        out = []
        for m, a, g, more, lay in zip(self.layers, self._acts, self._grads, self._options, layouts):
            if isinstance(m, Embedding):
                V, D = m.weight.shape
                scale, padding = more
                out.append(embedding_desc(DP_BF16 if g.dtype == torch.bfloat16 else DP_FP32, B=B, T=a.numel() // B, V=V,
                                          D=D, scale=scale, padding=padding, index_i64=a.dtype == torch.int64))
                continue
            hb = m.bias is not None
            if isinstance(m, LayerNorm):
                out.append(kept_desc(B=B, p=m.weight.numel(), has_bias=hb))
                continue
            if isinstance(m, nn.Linear):
                T = a.numel() // (B * m.in_features)
                out.append(layer_desc(DP_LINEAR, dtype, B=B, p=m.out_features, T=T, d=m.in_features, has_bias=hb))
            elif isinstance(m, nn.Conv1d):
                out.append(layer_desc(DP_CONV1D, dtype, B=B, p=m.out_channels, Cin=m.in_channels, H=1, W=a.shape[2],
                                      k=m.kernel_size[0], stride=m.stride[0], pad=m.padding[0], dil=m.dilation[0],
                                      has_bias=hb))
            elif isinstance(m, nn.Conv3d):
                out.append(layer_desc(DP_CONV3D, dtype, B=B, p=m.out_channels, Cin=m.in_channels, Z=a.shape[2],
                                      H=a.shape[3], W=a.shape[4], k=m.kernel_size[0], stride=m.stride[0],
                                      pad=m.padding[0], dil=m.dilation[0], has_bias=hb, layout=lay))
            else:
                out.append(layer_desc(DP_CONV2D, dtype, B=B, p=m.out_channels, Cin=m.in_channels, H=a.shape[2],
                                      W=a.shape[3], k=m.kernel_size[0], stride=m.stride[0], pad=m.padding[0],
                                      dil=m.dilation[0], has_bias=hb, layout=lay))
        return out

    def privatise(self, seed: int, stream=None):
        """Replace every layer's .grad by its privatised gradient; returns the flat vector."""
        import torch
        if any(a is None or (g is None and not isinstance(m, LayerNorm))
               for m, a, g in zip(self.layers, self._acts, self._grads)):
            raise RuntimeError("run the forward pass and loss.backward() first")
        B = self._acts[0].shape[0]
        if any(a.shape[0] != B for m, a in zip(self.layers, self._acts) if isinstance(m, (Embedding, LayerNorm))):
            raise ValueError(f"an embedding's tokens or a layer norm's inputs are not of {B} examples")
        # the type of A and G, which linear and conv layers share
        dt = next((a.dtype for m, a in zip(self.layers, self._acts) if not isinstance(m, (Embedding, LayerNorm))),
                  torch.float32)
        if dt not in (torch.bfloat16, torch.float32):
            raise ValueError(f"inputs of dtype {dt}: bf16 or fp32 only")
        dtype = DP_BF16 if dt == torch.bfloat16 else DP_FP32
        layouts = [self._layout(m, a) for m, a in zip(self.layers, self._acts)]
        # what the step's descriptors and buffers go by
        key = (B, dtype, self._acts[0].device, tuple(tuple(a.shape) for a in self._acts), tuple(layouts), tuple(
            (a.dtype, g.dtype, more) for m, a, g, more in zip(self.layers, self._acts, self._grads, self._options)
            if isinstance(m, Embedding)))
        if self._key != key:
            self._step = ClipStep(self._descs(B, dtype, layouts), C=self.C, sigma=self.sigma, per_layer=self.per_layer,
                                  norm_modes=[self.norm_mode] * len(self.layers), device=str(self._acts[0].device),
                                  keep_grads=self.keep_grads)
            self._key = key
        scale = float(B) if self.loss_reduction == "mean" else 1.0

        def times(g):
            return g * scale if scale != 1.0 else g
        inputs = []
        for m, a, g, lay in zip(self.layers, self._acts, self._grads, layouts):
            if isinstance(m, Embedding):
                inputs.append((a.contiguous(), times(g).contiguous()))
            elif isinstance(m, LayerNorm):
                inputs.append((times(a), None))
            else:
                inputs.append((self._as_layout(a, lay, dt), self._as_layout(times(g), lay, dt)))
        flat = self._step.run(inputs, seed=seed, stream=stream)
        for l, m in enumerate(self.layers):
            dW, db = self._step.layer_views(l)
            m.weight.grad = dW.view_as(m.weight).to(m.weight.dtype).clone()
            if getattr(m, "bias", None) is not None:
                m.bias.grad = db.to(m.bias.dtype).clone()
        self._acts = [None] * len(self.layers)
        self._grads = [None] * len(self.layers)
        return flat
