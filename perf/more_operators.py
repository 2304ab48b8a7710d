"""The trained ends of a private sequence model: embeddings and layer norms with their gradients and per-example
clipping, and the log probabilities that its answers are scored and distilled with -- the cases they are timed and
checked on, and their plain forms.

A private training step looks its tokens up, normalises between the linear layers, and clips both layers' gradients
per example beside the linear ones; the teacher's top alternatives and the scores of given tokens come from the
log probabilities.  `run` computes a case in elementary torch operations in 32 bits (own = False) or by the
package's operators (own = True); `exact` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One new token of a batch of sequences, scaled by sqrt(D): latency only.
        dict(name="embedding_one_token", op="embedding", dtype="bf16", B=64, T=1, V=50257, D=768, scaled=True,
             padded=False, mode="lookup"),
        # A training step: the lookup, and the whole weight's gradient in the weight's type.
        dict(name="embedding_train", op="embedding", dtype="bf16", B=32, T=512, V=50257, D=768, scaled=True,
             padded=True, mode="train"),
        # Private training, fp32, rows that no vector load fits, a padded batch with an empty example.
        dict(name="embedding_private_odd", op="embedding", dtype="fp32", B=16, T=250, V=1000, D=197, scaled=False,
             padded=True, mode="private"),
        # Private training on long documents over a large vocabulary: the largest.
        dict(name="embedding_private_long", op="embedding", dtype="bf16", B=64, T=4096, V=131072, D=1024,
             scaled=False, padded=False, mode="private"),
        # One new token of a batch of sequences: latency only.
        dict(name="layer_norm_one_token", op="layer_norm", dtype="bf16", B=64, T=1, D=768, bias=True, padded=False,
             mode="forward"),
        # A training step at the ViT-Base layer size of the framework's workloads.
        dict(name="layer_norm_vit_train", op="layer_norm", dtype="bf16", B=64, T=197, D=768, bias=True, padded=False,
             mode="train"),
        # Private training, fp32, an odd width, padded examples.
        dict(name="layer_norm_private_odd", op="layer_norm", dtype="fp32", B=16, T=250, D=1001, bias=True,
             padded=True, mode="private"),
        # A wide decoder's training step over long sequences, no bias.
        dict(name="layer_norm_wide_train", op="layer_norm", dtype="bf16", B=4, T=8191, D=4096, bias=False,
             padded=False, mode="train"),
        # Serving: one token of eight sequences, its score and twenty alternatives.
        dict(name="logprobs_one_token", op="logprobs", dtype="bf16", B=8, T=1, V=131072, K=20, tau=1.0, grad=False),
        # A few rows over a small vocabulary, fp32, with the gradient: latency only.
        dict(name="logprobs_small_fp32", op="logprobs", dtype="fp32", B=4, T=31, V=1000, K=16, tau=2.0, grad=True),
        # A teacher's top alternatives over a held-out batch, an odd vocabulary (rows not 16-byte aligned).
        dict(name="logprobs_teacher", op="logprobs", dtype="bf16", B=32, T=128, V=50257, K=50, tau=1.0, grad=False),
        # Training on scored answers with an entropy term, a large odd vocabulary: gradient of both.
        dict(name="logprobs_train", op="logprobs", dtype="bf16", B=8, T=1024, V=131071, K=0, tau=1.0, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "layer_norm", "logprobs"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    most = 1 if dtype == "bf16" else 2   # an fp32 case has half the elements
    if op == "embedding":
        D = rng.choice([64, 128, 197, 250, 512, 768, 1024, 1000, 1280, 2048, _log_int(rng, 16, 2048)])
        V = min(_log_int(rng, 300, 200000), (1 << 27) // (most * D))
        T = _log_int(rng, 1, 8192)
        B = max(1, min(_log_int(rng, 1, 1024), (1 << 28) // (most * T * D)))
        return dict(op=op, dtype=dtype, B=B, T=T, V=V, D=D, scaled=rng.random() < 0.5,
                    padded=T > 1 and rng.random() < 0.5, mode=rng.choice(["lookup", "train", "private", "private"]))
    if op == "layer_norm":
        D = rng.choice([64, 128, 256, 768, 1001, 1024, 1536, 2048, 4096, 5120, 8192, _log_int(rng, 16, 12288)])
        T = _log_int(rng, 1, 8192)
        B = max(1, min(_log_int(rng, 1, 1024), 4 * 8191 * 4096 // (most * T * D)))
        return dict(op=op, dtype=dtype, B=B, T=T, D=D, bias=rng.random() < 0.8, padded=T > 1 and rng.random() < 0.4,
                    mode=rng.choice(["forward", "train", "train", "private"]))
    V = _log_int(rng, 300, 200000)
    N = max(1, min(_log_int(rng, 1, 8192), 8 * 1024 * 131071 // (2 * most * V)))
    T = min(N, _log_int(rng, 1, 1024))
    return dict(op=op, dtype=dtype, B=max(1, N // T), T=T, V=V, K=rng.choice([0, 1, 5, 20, 50, 64, 100]),
                tau=rng.choice([1.0, 1.0, 2.0, 0.7]), grad=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------- inputs
def _lengths(B, T):
    """Lengths of a padded batch: spread evenly from the full length down to an empty example."""
    return [T - (T * i) // max(1, B - 1) for i in range(B)]


def _scale(case):
    return math.sqrt(case["D"]) if case["scaled"] else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, T = _DT[case["dtype"]], case["B"], case["T"]
    new = dict(generator=g, device="cuda")

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, **new) * std).to(dt)

    st = dict(case=case)
    there = torch.ones(B, T, dtype=torch.bool, device="cuda")
    if case.get("padded"):
        lens = torch.tensor(_lengths(B, T), device="cuda")[torch.randperm(B, **new)]
        there = torch.arange(T, device="cuda")[None, :] < lens[:, None]
    if case["op"] == "embedding":
        V, D = case["V"], case["D"]
        # tokens as frequent as one over their rank, the ranks scattered over the vocabulary
        rank = torch.exp(torch.rand(B, T, dtype=torch.float64, **new) * math.log(V + 1)).long().clamp(1, V) - 1
        tokens = (rank * 7919) % V
        st["padding"] = None
        if case["padded"]:
            st["padding"] = V - 1
            tokens = torch.where(there, tokens, torch.full_like(tokens, V - 1))
        st["tokens"] = tokens.to(torch.int32).contiguous()
        if case["mode"] != "private":
            st["weight"] = normal(V, D, std=0.02)
        if case["mode"] != "lookup":
            st["dy"] = normal(B, T, D, std=0.01)
        if case["mode"] == "private":
            st["C"] = 0.01 * math.sqrt(0.7 * T * D)   # some examples below the bound, some above
            if own:
                import example_gradient_clipping_gb300 as dp
                desc = dp.embedding_desc(dp.DP_BF16 if case["dtype"] == "bf16" else dp.DP_FP32, B=B, T=T, V=V, D=D,
                                         scale=_scale(case), padding=st["padding"])
                st["step"] = dp.ClipStep([desc], C=st["C"], sigma=0.0)
        return st
    if case["op"] == "layer_norm":
        D = case["D"]
        # channels of their own mean and size, a few of them large
        size = torch.exp(0.5 * torch.randn(D, **new))
        size[torch.randint(0, D, (max(1, D // 256),), **new)] *= 20.0
        st["x"] = (torch.randn(B, T, D, **new) * size + 0.3 * torch.randn(D, **new)).to(dt)
        st["weight"] = (1.0 + 0.1 * torch.randn(D, **new)).to(dt)
        st["bias"] = normal(D, std=0.1) if case["bias"] else None
        if case["mode"] != "forward":
            st["dy"] = torch.where(there[..., None], normal(B, T, D, std=0.01), torch.zeros((), dtype=dt, device="cuda"))
        if case["mode"] == "private":
            st["C"] = 0.01 * math.sqrt(0.7 * T * D * (2 if case["bias"] else 1))
            if own:
                import example_gradient_clipping_gb300 as dp
                st["step"] = dp.ClipStep([dp.kept_desc(B=B, p=D, has_bias=case["bias"])], C=st["C"], sigma=0.0)
        return st
    V = case["V"]
    logits = torch.randn(B, T, V, **new) * 2.0
    tokens = torch.randint(0, V, (B, T, 1), **new)
    logits.scatter_add_(2, tokens, torch.rand(B, T, 1, **new) * 12.0)   # the given tokens are likely ones
    st["logits"] = logits.to(dt)
    del logits
    lens = torch.tensor([max(n, (T + 1) // 2) for n in _lengths(B, T)], device="cuda")[torch.randperm(B, **new)]
    there = torch.arange(T, device="cuda")[None, :] < lens[:, None]
    st["tokens"] = torch.where(there, tokens.squeeze(-1), -1).to(torch.int32).contiguous()   # -1: no token given
    if case["grad"]:
        st["d_logprob"] = torch.randn(B, T, **new) * there
        st["d_entropy"] = -0.1 * torch.rand(B, T, **new) * there
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _factors_plain(sq, C):
    n = torch.sqrt(sq)
    return torch.where(n <= C, torch.ones_like(n), C / n)


def _embedding_plain(case, st):
    V, D, mode, s = case["V"], case["D"], case["mode"], _scale(case)
    tokens = st["tokens"].long()
    out = ()
    if mode != "private":
        out = ((st["weight"][tokens].float() * s).to(st["weight"].dtype),)
        if mode == "lookup":
            return out[0]
    dy = st["dy"].float()
    if st["padding"] is not None:
        dy = dy * (tokens != st["padding"]).unsqueeze(-1)
    total = torch.zeros(V, D, dtype=torch.float32, device="cuda")
    if mode == "train":
        return out + (total.index_add_(0, tokens.flatten(), dy.view(-1, D)).mul_(s).to(st["weight"].dtype),)
    sq = torch.empty(case["B"], dtype=torch.float32, device="cuda")
    for i in range(case["B"]):
        one = total.zero_().index_add_(0, tokens[i], dy[i])
        sq[i] = (one * one).sum() * (s * s)
    c = _factors_plain(sq, st["C"])
    dw = total.zero_().index_add_(0, tokens.flatten(), (dy * c[:, None, None]).view(-1, D)).mul_(s)
    return sq, c, dw


def _layer_norm_plain(case, st):
    x, w = st["x"].float(), st["weight"].float()
    mean = x.mean(dim=-1, keepdim=True)
    xhat = x - mean
    rstd = torch.rsqrt((xhat * xhat).mean(dim=-1, keepdim=True) + 1e-5)
    xhat = xhat.mul_(rstd)
    y = xhat * w
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = y.to(st["x"].dtype)
    if case["mode"] == "forward":
        return y
    dy = st["dy"].float()
    g = dy * w
    dx = ((g - g.mean(dim=-1, keepdim=True) - xhat * (g * xhat).mean(dim=-1, keepdim=True)) * rstd).to(st["x"].dtype)
    dw, db = (dy * xhat).sum(dim=1), dy.sum(dim=1)
    if case["mode"] == "train":
        dw, db = dw.sum(dim=0).to(st["weight"].dtype), db.sum(dim=0).to(st["weight"].dtype)
        return (y, dx, dw, db) if case["bias"] else (y, dx, dw)
    each = torch.cat([dw, db], dim=1) if case["bias"] else dw
    sq = (each * each).sum(dim=1)
    c = _factors_plain(sq, st["C"])
    return y, dx, sq, c, (each * c[:, None]).sum(dim=0)


def _logprobs_plain(case, st):
    tau, K = case["tau"], case["K"]
    z = st["logits"].to(torch.float32, copy=True)   # (its own: the inputs stay as they are)
    if K:
        v, i = torch.sort(z, dim=-1, descending=True, stable=True)
        top, top_index = v[..., :K] / tau, i[..., :K].to(torch.int32)
        del v, i
    z = z.div_(tau)
    m = z.amax(dim=-1, keepdim=True)
    z = z.sub_(m)
    e = torch.exp(z)
    n = e.sum(dim=-1, keepdim=True)
    log_n = torch.log(n)
    p = e.div_(n)
    given = st["tokens"] >= 0
    y = st["tokens"].clamp(min=0).long().unsqueeze(-1)
    logprob = torch.where(given, (torch.gather(z, 2, y) - log_n).squeeze(-1), 0.0)
    z = z.sub_(log_n)   # log p
    entropy = -(p * z).sum(dim=-1)
    out = (logprob, entropy)
    if K:
        out = out + (top - m - log_n, top_index)
    if case["grad"]:
        dl = torch.where(given, st["d_logprob"], 0.0).unsqueeze(-1)
        dz = z.add_(entropy.unsqueeze(-1)).mul_(-st["d_entropy"].unsqueeze(-1)).sub_(dl).mul_(p)
        dz = dz.scatter_add_(2, y, dl).mul_(1.0 / tau)
        out = out + (dz.to(st["logits"].dtype),)
    return out


def run(state):
    case, st = state["case"], state
    if not own:
        return {"embedding": _embedding_plain, "layer_norm": _layer_norm_plain, "logprobs": _logprobs_plain}[case["op"]](case, st)
    import example_gradient_clipping_gb300 as dp
    if case["op"] == "embedding":
        if case["mode"] == "private":
            step, inputs = st["step"], [(st["tokens"], st["dy"])]
            step.norms(inputs)
            step.factors_()
            step.sums(inputs)
            return step.sqnorms[0], step.factors[0], step.grad.view(case["V"], case["D"])
        y = dp.embedding(st["tokens"], st["weight"], scale=_scale(case), padding=st["padding"])
        if case["mode"] == "lookup":
            return y
        return y, dp.embedding_backward(st["tokens"], st["dy"], case["V"], scale=_scale(case), padding=st["padding"],
                                        dtype=st["weight"].dtype)
    if case["op"] == "layer_norm":
        if case["mode"] == "forward":
            return dp.layer_norm(st["x"], st["weight"], st["bias"])
        y, mean, rstd = dp.layer_norm_forward(st["x"], st["weight"], st["bias"])
        if case["mode"] == "train":
            dx, dw, db = dp.layer_norm_backward(st["dy"], st["x"], st["weight"], mean, rstd, bias=case["bias"])
            return (y, dx, dw, db) if case["bias"] else (y, dx, dw)
        dx, each = dp.layer_norm_backward(st["dy"], st["x"], st["weight"], mean, rstd, bias=case["bias"], per_example=True)
        step, inputs = st["step"], [(each, None)]
        step.norms(inputs)
        step.factors_()
        step.sums(inputs)
        return y, dx, step.sqnorms[0], step.factors[0], step.grad
    logprob, entropy, stats, top, top_index = dp.token_logprobs_forward(st["logits"], st["tokens"], top=case["K"],
                                                                        temperature=case["tau"])
    out = (logprob, entropy) + ((top, top_index) if case["K"] else ())
    if case["grad"]:
        out = out + (dp.token_logprobs_backward(st["logits"], st["tokens"], stats, entropy, st["d_logprob"],
                                                st["d_entropy"], temperature=case["tau"]),)
    return out


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    es, B, T = _ES[case["dtype"]], case["B"], case["T"]
    if case["op"] == "embedding":
        V, D = case["V"], case["D"]
        n = sum(_lengths(B, T)) if case["padded"] else B * T   # rows with a gradient
        p = np.log1p(1.0 / np.arange(1, V + 1)) / math.log(V + 1)
        met = float(-np.expm1(n * np.log1p(-p)).sum())         # expected different tokens
        rows, tokens = B * T * D * es, B * T * 4
        if case["mode"] == "lookup":
            return {"bytes": rows + met * D * es + tokens, "flops": B * T * D if case["scaled"] else 0}
        if case["mode"] == "train":   # the lookup, then the gradient's rows in and the whole weight's gradient out
            return {"bytes": rows + met * D * es + n * D * es + V * D * es + tokens, "flops": (2 * n + B * T) * D}
        return {"bytes": n * D * es + V * D * 4 + tokens + B * 8, "flops": 5 * n * D}
    if case["op"] == "layer_norm":
        n, D = B * T, case["D"]
        k = 2 if case["bias"] else 1
        if case["mode"] == "forward":
            return {"bytes": 2 * n * D * es + k * D * es, "flops": 7 * n * D}
        if case["mode"] == "train":   # x and dy in, y and dx out
            return {"bytes": 4 * n * D * es + 2 * k * D * es, "flops": 20 * n * D}
        return {"bytes": 4 * n * D * es + k * D * (es + 4) + B * 8, "flops": 20 * n * D + 4 * B * k * D}
    n, V, K = B * T, case["V"], case["K"]
    small = n * (4 + 8 + 8 * K)
    if case["grad"]:
        return {"bytes": 2 * n * V * es + small + 8 * n, "flops": 14 * n * V}
    return {"bytes": n * V * es + small, "flops": 6 * n * V}


# ---------------------------------------------------------------------------------------------------- 64 bits
def _clip(norms, C):
    return torch.clamp(C / norms.clamp(min=1e-300), max=1.0)


def _exact_embedding(case, st):
    V, D, mode, s = case["V"], case["D"], case["mode"], _scale(case)
    new = dict(dtype=torch.float64, device="cuda")
    out = ()
    if mode != "private":
        y = torch.empty(case["B"], case["T"], D, **new)
        for i in range(case["B"]):
            y[i] = torch.index_select(st["weight"], 0, st["tokens"][i].long()).double() * s
        out = (y,)
        if mode == "lookup":
            return y
    total = torch.zeros(V, D, **new)
    sq, c = torch.zeros(case["B"], **new), torch.ones(case["B"], **new)
    for i in range(case["B"]):
        t = st["tokens"][i]
        keep = torch.ones_like(t, dtype=torch.bool) if st["padding"] is None else t != st["padding"]
        which, back = torch.unique(t[keep], return_inverse=True)
        one = torch.zeros(len(which), D, **new).index_add_(0, back, st["dy"][i][keep].double()) * s
        if mode == "private":
            sq[i] = one.pow(2).sum()
            c[i] = _clip(sq[i].sqrt(), st["C"])
        total[which.long()] += c[i] * one
    return out + (total,) if mode == "train" else (sq, c, total)


def _exact_layer_norm(case, st):
    B, T, D = case["B"], case["T"], case["D"]
    new = dict(dtype=torch.float64, device="cuda")
    w = st["weight"].double()
    b = st["bias"].double() if st["bias"] is not None else torch.zeros(D, **new)
    y = torch.empty(B, T, D, **new)
    grad = case["mode"] != "forward"
    dx = torch.empty(B, T, D, **new) if grad else None
    k = 2 if case["bias"] else 1
    each = torch.zeros(B, k * D, **new)
    for i in range(B):
        x = st["x"][i].double()
        var, mu = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        sd = torch.sqrt(var + 1e-5)
        h = (x - mu) / sd
        y[i] = torch.addcmul(b, h, w)
        if not grad:
            continue
        g = st["dy"][i].double()
        u = g * w
        # off u's parts along the ones and along h
        dx[i] = (u - u.sum(1, keepdim=True) / D - h * (torch.einsum("td,td->t", u, h)[:, None] / D)) / sd
        each[i, :D] = torch.einsum("td,td->d", g, h)
        if case["bias"]:
            each[i, D:] = g.sum(0)
    if not grad:
        return y
    if case["mode"] == "train":
        t = each.sum(0)
        return (y, dx, t[:D], t[D:]) if case["bias"] else (y, dx, t)
    n = torch.linalg.vector_norm(each, dim=1)
    c = _clip(n, st["C"])
    return y, dx, n * n, c, c @ each


def _exact_logprobs(case, st):
    B, T, V, K, tau = case["B"], case["T"], case["V"], case["K"], case["tau"]
    new = dict(dtype=torch.float64, device="cuda")
    logprob, entropy = torch.zeros(B, T, **new), torch.zeros(B, T, **new)
    top = torch.empty(B, T, K, **new)
    top_index = torch.empty(B, T, K, dtype=torch.int32, device="cuda")
    grad = torch.empty(B, T, V, **new) if case["grad"] else None
    for b in range(B):
        for t in range(0, T, 256):
            at = slice(t, min(T, t + 256))
            z = st["logits"][b, at]
            lp = torch.log_softmax(z.double() / tau, dim=1)
            p = torch.exp(lp)
            h = -torch.einsum("tv,tv->t", p, lp)
            entropy[b, at] = h
            y = st["tokens"][b, at].long()
            r = torch.nonzero(y >= 0).flatten()
            logprob[b, at][r] = lp[r, y[r]]
            if K:
                order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :K]
                top_index[b, at] = order.to(torch.int32)
                top[b, at] = torch.gather(lp, 1, order)
            if case["grad"]:
                up = torch.where(y >= 0, st["d_logprob"][b, at].double(), 0.0)
                d = -up[:, None] * p - st["d_entropy"][b, at].double()[:, None] * p * (lp + h[:, None])
                d[r, y[r]] += up[r]
                grad[b, at] = d / tau
    return (logprob, entropy) + ((top, top_index) if K else ()) + ((grad,) if case["grad"] else ())


def exact(case, seed):
    st = prepare(case, seed)
    return {"embedding": _exact_embedding, "layer_norm": _exact_layer_norm, "logprobs": _exact_logprobs}[case["op"]](case, st)
