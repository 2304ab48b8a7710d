"""The sequence operators around the clipped layers: rotary positions, attention with its gradient, and the
distillation loss with its gradient -- the cases they are timed and checked on, and their plain forms.

A private training step of a sequence model runs them between the linear layers whose per-example gradients are
clipped.  `run` computes a case in elementary torch operations in 32 bits (own = False) or by the package's
operators (own = True); `exact` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}
NEG = -float("inf")


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One new position of a batch of sequences: latency only.
        dict(name="rotary_one_token", op="rotary", dtype="bf16", B=64, T=1, Hq=12, Hk=12, D=64, R=64, layout="half",
             P=2048, scaling="none", inverse=False),
        # Q and K read from one packed projection of a ViT-Base-sized layer (T = 197), fp32.
        dict(name="rotary_packed_fp32", op="rotary", dtype="fp32", B=64, T=197, Hq=12, Hk=12, D=64, R=64,
             layout="interleaved", P=197, scaling="none", inverse=False, packed=True),
        # Gradient direction, half of each head rotated, shared key heads, a context stretched past its trained length.
        dict(name="rotary_long_grad", op="rotary", dtype="bf16", B=4, T=8191, Hq=32, Hk=8, D=128, R=64, layout="half",
             P=131072, scaling="parts", inverse=True),
        # Short ragged sequences, a padded batch with an empty example: evaluation.
        dict(name="attention_short", op="attention", dtype="bf16", B=4, T=33, S=33, Hq=12, Hk=12, D=64, causal=True,
             window=0, ragged=True, grad=False),
        # A training step's attention at the ViT-Base layer size of the framework's workloads.
        dict(name="attention_vit_train", op="attention", dtype="bf16", B=64, T=197, S=197, Hq=12, Hk=12, D=64,
             causal=False, window=0, ragged=False, grad=True),
        # fp32 training of short sequences (the framework's fp32 path), ragged.
        dict(name="attention_fp32_train", op="attention", dtype="fp32", B=16, T=250, S=250, Hq=12, Hk=12, D=64,
             causal=True, window=0, ragged=True, grad=True),
        # A decoder's training step: causal, four query heads to a key head.
        dict(name="attention_causal_train", op="attention", dtype="bf16", B=2, T=4096, S=4096, Hq=16, Hk=4, D=128,
             causal=True, window=0, ragged=False, grad=True),
        # The longest: one example of 8192 tokens, forward only (evaluation of a long document).
        dict(name="attention_long", op="attention", dtype="bf16", B=1, T=8192, S=8192, Hq=32, Hk=8, D=128, causal=True,
             window=0, ragged=False, grad=False),
        # A few rows over a small vocabulary, fp32: latency only.
        dict(name="distill_small_fp32", op="distill", dtype="fp32", B=4, T=31, V=1000, K=16, tau=2.0, alpha=0.5,
             grad=True),
        # An odd vocabulary (rows not 16-byte aligned), padded examples, labels mixed in.
        dict(name="distill_odd_vocab", op="distill", dtype="bf16", B=16, T=128, V=50257, K=32, tau=2.0, alpha=0.3,
             grad=True),
        # The loss of a held-out batch, per example and per token, no gradient.
        dict(name="distill_eval", op="distill", dtype="bf16", B=32, T=128, V=32768, K=50, tau=1.0, alpha=0.0,
             grad=False),
        # A large vocabulary at a training batch.
        dict(name="distill_large_vocab", op="distill", dtype="bf16", B=8, T=1024, V=131072, K=64, tau=1.0, alpha=0.0,
             grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "attention", "attention", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "rotary":
        D = rng.choice([32, 40, 64, 80, 96, 128])
        Hk = rng.choice([1, 2, 4, 8, 12])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        T = _log_int(rng, 1, 4096)
        B = max(1, min(_log_int(rng, 1, 256), (1 << 27) // (T * (Hq + Hk) * D)))
        packed = Hq == Hk and rng.random() < 0.3
        return dict(op="rotary", dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, D // 2]),
                    layout=rng.choice(["half", "interleaved"]), P=max(T, _log_int(rng, 64, 131072)),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), inverse=rng.random() < 0.5, packed=packed)
    if kind == "attention":
        D = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        grad = rng.random() < 0.6
        T = _log_int(rng, 1, 3000 if dtype == "bf16" else 1500)
        S = T if rng.random() < 0.7 else _log_int(rng, 1, 3000 if dtype == "bf16" else 1500)
        most = (1 << 28) if dtype == "bf16" else (1 << 26)   # score entries of the batch
        B = max(1, min(_log_int(rng, 1, 64), most // (Hq * T * S)))
        causal = rng.random() < 0.6
        return dict(op="attention", dtype=dtype, B=B, T=T, S=S, Hq=Hq, Hk=Hk, D=D, causal=causal,
                    window=_log_int(rng, 1, max(2, S)) if causal and rng.random() < 0.25 else 0,
                    ragged=rng.random() < 0.5, grad=grad)
    V = _log_int(rng, 500, 200000)
    N = max(2, min(_log_int(rng, 2, 8192), (1 << 29) // V))
    T = min(N, _log_int(rng, 1, 512))
    return dict(op="distill", dtype=dtype, B=max(1, N // T), T=T, V=V, K=min(_log_int(rng, 1, 128), V // 2),
                tau=rng.choice([1.0, 1.0, 2.0, 4.0]), alpha=rng.choice([0.0, 0.0, 0.3, 1.0]), grad=rng.random() < 0.7)


# ---------------------------------------------------------------------------------------------------- inputs
def _lengths(B, T):
    """Lengths of a padded batch: spread evenly from the full length down to an empty example."""
    return [T - (T * i) // max(1, B - 1) for i in range(B)]


def _frequencies(case):
    """Angles per position of each rotated pair, and the table's magnitude (64 bits)."""
    R, s, theta = case["R"], 8.0, 10000.0
    j = np.arange(R // 2, dtype=np.float64)
    if case["scaling"] == "base":
        theta = theta * s ** (R / (R - 2)) if R > 2 else theta
    f = theta ** (-2.0 * j / R)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "parts":
        turns = 4096.0 * f / (2.0 * math.pi)
        g = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * ((1.0 - g) / s + g), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _table(case):
    f, mag = _frequencies(case)
    a = torch.arange(case["P"], dtype=torch.float64, device="cuda")[:, None] * torch.tensor(f, device="cuda")[None, :]
    return torch.cat([torch.cos(a) * mag, torch.sin(a) * mag], dim=1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    B, T = case["B"], case["T"]
    st = dict(case=case)
    if case["op"] == "rotary":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        if case.get("packed"):
            qkv = normal(B, T, 3, Hq, D)
            st["q"], st["k"] = qkv[:, :, 0], qkv[:, :, 1]
        else:
            st["q"], st["k"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
        # the table a program builds once, and where each example starts in its context
        st["table"] = _table(case).float()
        start = torch.randint(0, case["P"] - T + 1, (B, 1), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(T, device="cuda")[None, :]).to(torch.int32).contiguous()
        return st
    if case["op"] == "attention":
        S, Hq, Hk, D = case["S"], case["Hq"], case["Hk"], case["D"]
        st["q"], st["k"], st["v"] = normal(B, T, Hq, D), normal(B, S, Hk, D), normal(B, S, Hk, D)
        st["q_lens"] = st["k_lens"] = None
        if case["ragged"]:
            order = torch.randperm(B, generator=g, device="cuda")
            st["q_lens"] = torch.tensor(_lengths(B, T), dtype=torch.int32, device="cuda")[order].contiguous()
            st["k_lens"] = torch.tensor(_lengths(B, S), dtype=torch.int32, device="cuda")[order].contiguous()
        if case["grad"]:
            st["do"] = normal(B, T, Hq, D, std=0.01)
        return st
    V, K = case["V"], case["K"]
    logits = torch.randn(B, T, V, generator=g, device="cuda") * 2.0
    base = torch.randint(0, V, (B, T, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, V // K), (B, T, 1), generator=g, device="cuda")
    idx = (base + step * torch.arange(K, device="cuda")) % V
    teacher = torch.sort(torch.randn(B, T, K, generator=g, device="cuda") * 2.0 + 6.0, dim=-1, descending=True).values
    logits.scatter_add_(2, idx, 0.7 * teacher)   # a student that has learnt some of it
    st["logits"] = logits.to(dt)
    del logits
    have = torch.randint(max(1, K // 2), K + 1, (B, T, 1), generator=g, device="cuda")
    st["idx"] = torch.where(torch.arange(K, device="cuda") < have, idx, -1).to(torch.int32)
    st["teacher"] = teacher.to(dt)
    st["labels"] = torch.randint(0, V, (B, T), generator=g, device="cuda").to(torch.int32) if case["alpha"] > 0 else None
    lens = torch.tensor(_lengths(B, T), device="cuda")[torch.randperm(B, generator=g, device="cuda")]
    st["weights"] = (torch.arange(T, device="cuda")[None, :] < torch.clamp(lens, min=T // 2)[:, None]).float()
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _rotate_plain(case, x, cs):
    R, dt = case["R"], x.dtype
    c, s = cs[..., : R // 2].unsqueeze(2), cs[..., R // 2:].unsqueeze(2)
    if case["inverse"]:
        s = -s
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., : R // 2], y[..., R // 2: R]
        r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([r, y[..., R:]], dim=-1).to(dt)


def _visible(case, st, device):
    """[B, T, S] truth values: which keys each query sees."""
    B, T, S = case["B"], case["T"], case["S"]
    lq = st["q_lens"].long() if st["q_lens"] is not None else torch.full((B,), T, device=device)
    lk = st["k_lens"].long() if st["k_lens"] is not None else torch.full((B,), S, device=device)
    t = torch.arange(T, device=device)[None, :, None]
    j = torch.arange(S, device=device)[None, None, :]
    see = (t < lq[:, None, None]) & (j < lk[:, None, None])
    last = t + (lk - lq)[:, None, None]
    if case["causal"]:
        see = see & (j <= last)
    if case["window"]:
        see = see & (j > last - case["window"])
    return see


def _attention_plain(case, st):
    B, T, S, Hq, Hk, D = (case[n] for n in ("B", "T", "S", "Hq", "Hk", "D"))
    G, dt, scale = Hq // Hk, st["q"].dtype, 1.0 / math.sqrt(D)
    q = st["q"].float().permute(0, 2, 1, 3).reshape(B, Hk, G * T, D)
    k, v = st["k"].float().permute(0, 2, 1, 3), st["v"].float().permute(0, 2, 1, 3)
    see = _visible(case, st, q.device)[:, None, None]
    s = (q @ k.transpose(-1, -2)).mul_(scale).view(B, Hk, G, T, S).masked_fill_(~see, NEG)
    top = s.amax(dim=-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp(s.sub_(top))
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + top).view(B, Hq, T)
    p = (p / torch.where(total == 0, torch.ones_like(total), total)).view(B, Hk, G * T, S)
    del s
    o = p @ v

    def heads(x, n):
        return x.reshape(B, n, -1, D).permute(0, 2, 1, 3).contiguous().to(dt)

    if not case["grad"]:
        return heads(o, Hq), lse
    do = st["do"].float().permute(0, 2, 1, 3).reshape(B, Hk, G * T, D)
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p).mul_(scale)
    return heads(o, Hq), lse, heads(ds @ k, Hq), heads(ds.transpose(-1, -2) @ q, Hk), heads(dv, Hk)


def _distill_plain(case, st):
    tau, alpha, w = case["tau"], case["alpha"], st["weights"]
    z = st["logits"].float()
    have = st["idx"] >= 0
    idx = st["idx"].clamp(min=0).long()
    t = torch.where(have, st["teacher"].float() / tau, torch.full_like(st["teacher"], NEG, dtype=torch.float32))
    p = torch.exp(t - t.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)

    def soft(u):
        m = u.amax(dim=-1, keepdim=True)
        e = torch.exp(u - m)
        n = e.sum(dim=-1, keepdim=True)
        return m + torch.log(n), e.div_(n)

    lse, q = soft(z / tau)
    logp = torch.where(p > 0, torch.log(torch.where(p > 0, p, torch.ones_like(p))), torch.zeros_like(p))
    row = (1.0 - alpha) * tau * tau * (p * (logp - torch.gather(z, 2, idx) / tau + lse)).sum(dim=-1)
    grad = q.mul_((1.0 - alpha) * tau).scatter_add_(2, idx, p * (-(1.0 - alpha) * tau)) if case["grad"] else None
    if alpha > 0:
        lse1, q1 = soft(z)
        y = st["labels"].long().unsqueeze(-1)
        row = row + alpha * (lse1 - torch.gather(z, 2, y)).squeeze(-1)
        if case["grad"]:
            grad = grad.add_(q1, alpha=alpha).scatter_add_(2, y, torch.full_like(y, -alpha, dtype=torch.float32))
    row = row * w
    loss = row.sum(dim=-1)
    return (loss, grad.mul_(w.unsqueeze(-1)).to(st["logits"].dtype)) if case["grad"] else (loss, row)


def run(state):
    case, st = state["case"], state
    if own:
        import example_gradient_clipping_gb300 as dp
        if case["op"] == "rotary":
            return dp.rotary(st["q"], st["k"], st["table"], positions=st["positions"],
                             interleaved=case["layout"] == "interleaved", inverse=case["inverse"])
        if case["op"] == "attention":
            kw = dict(causal=case["causal"], window=case["window"], q_lens=st["q_lens"], k_lens=st["k_lens"])
            o, lse = dp.attention_forward(st["q"], st["k"], st["v"], **kw)
            if not case["grad"]:
                return o, lse
            return (o, lse) + dp.attention_backward(st["q"], st["k"], st["v"], o, lse, st["do"], **kw)
        kw = dict(labels=st["labels"], weights=st["weights"], temperature=case["tau"], alpha=case["alpha"])
        if case["grad"]:
            return dp.distill_loss_and_grad(st["logits"], st["idx"], st["teacher"], **kw)
        return dp.distill_loss(st["logits"], st["idx"], st["teacher"], **kw)
    if case["op"] == "rotary":
        cs = st["table"][st["positions"].long()]
        return _rotate_plain(case, st["q"], cs), _rotate_plain(case, st["k"], cs)
    if case["op"] == "attention":
        return _attention_plain(case, st)
    return _distill_plain(case, st)


# ---------------------------------------------------------------------------------------------------- work
def _pairs(case):
    """Query-key pairs that some query sees, over the batch (one head)."""
    n = 0
    lq = _lengths(case["B"], case["T"]) if case["ragged"] else [case["T"]] * case["B"]
    lk = _lengths(case["B"], case["S"]) if case["ragged"] else [case["S"]] * case["B"]
    for a, b in zip(lq, lk):
        last = np.arange(a) + (b - a)
        hi = np.minimum(last, b - 1) if case["causal"] else np.full(a, b - 1)
        lo = np.maximum(last - case["window"] + 1, 0) if case["window"] else np.zeros(a, dtype=np.int64)
        n += int(np.maximum(hi - lo + 1, 0).sum())
    return n


def work(case):
    es, B, T = _ES[case["dtype"]], case["B"], case["T"]
    if case["op"] == "rotary":
        n = B * T * (case["Hq"] + case["Hk"])
        # each row in and out, its position; the table's rows once for the positions met
        return {"bytes": 2 * n * case["D"] * es + B * T * 4 + min(case["P"], B * T) * case["R"] * 4,
                "flops": 3 * n * case["R"]}
    if case["op"] == "attention":
        S, Hq, Hk, D = case["S"], case["Hq"], case["Hk"], case["D"]
        q, kv, lse = B * T * Hq * D * es, 2 * B * S * Hk * D * es, B * T * Hq * 4
        pairs = _pairs(case) * Hq
        if case["grad"]:   # reads q, k, v, do; writes o, lse, dq, dk, dv
            return {"bytes": 4 * q + 2 * kv + lse, "flops": 14 * D * pairs}
        return {"bytes": 2 * q + kv + lse, "flops": 4 * D * pairs}
    V, K = case["V"], case["K"]
    lens = [max(n, T // 2) for n in _lengths(B, T)]
    rows = sum(lens)   # rows of weight 0 need not be read, their gradient is still written
    small = B * T * (K * (4 + es) + 8) + B * 4
    return {"bytes": rows * V * es + (B * T * V * es if case["grad"] else 0) + small,
            "flops": rows * V * ((8 if case["grad"] else 4) * (2 if case["alpha"] > 0 else 1))}


# ---------------------------------------------------------------------------------------------------- 64 bits
def _exact_rotary(case, st):
    f, mag = _frequencies(case)
    R = case["R"]
    angle = st["positions"].double().unsqueeze(-1) * torch.tensor(f, device="cuda")
    turn = torch.polar(torch.full_like(angle, mag), -angle if case["inverse"] else angle).unsqueeze(2)
    out = []
    for x in (st["q"], st["k"]):
        y = x.double().clone()
        if case["layout"] == "half":
            z = torch.complex(y[..., : R // 2].contiguous(), y[..., R // 2: R].contiguous()) * turn
            y[..., : R // 2], y[..., R // 2: R] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * turn
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_attention(case, st):
    """Example by example and head by head, over the keys that exist; O(T S) memory of one head."""
    B, T, S, Hq, Hk, D = (case[n] for n in ("B", "T", "S", "Hq", "Hk", "D"))
    new = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(B, T, Hq, D, **new), torch.full((B, Hq, T), NEG, **new)
    dq, dk, dv = torch.zeros(B, T, Hq, D, **new), torch.zeros(B, S, Hk, D, **new), torch.zeros(B, S, Hk, D, **new)
    lq = st["q_lens"].tolist() if st["q_lens"] is not None else [T] * B
    lk = st["k_lens"].tolist() if st["k_lens"] is not None else [S] * B
    for b in range(B):
        a, n = lq[b], lk[b]
        if a == 0 or n == 0:
            continue
        gap = torch.arange(n, device="cuda")[None, :] - (torch.arange(a, device="cuda")[:, None] + (n - a))
        hidden = torch.zeros(a, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= gap > 0
        if case["window"]:
            hidden |= gap <= -case["window"]
        for h in range(Hq):
            kh = h * Hk // Hq
            q, k, v = st["q"][b, :a, h].double(), st["k"][b, :n, kh].double(), st["v"][b, :n, kh].double()
            x = q.mm(k.t()) / math.sqrt(D)
            x[hidden] = NEG
            y = torch.logsumexp(x, dim=1)
            p = torch.nan_to_num(torch.exp(x - y[:, None]), nan=0.0)
            lse[b, h, :a] = y
            o[b, :a, h] = p.mm(v)
            if case["grad"]:
                g = st["do"][b, :a, h].double()
                dv[b, :n, kh] += p.t().mm(g)
                e = g.mm(v.t())
                e = p * (e - (p * e).sum(dim=1, keepdim=True)) / math.sqrt(D)
                dq[b, :a, h] = e.mm(k)
                dk[b, :n, kh] += e.t().mm(q)
    return (o, lse, dq, dk, dv) if case["grad"] else (o, lse)


def _exact_distill(case, st):
    B, T, V, tau, alpha = case["B"], case["T"], case["V"], case["tau"], case["alpha"]
    rows = torch.zeros(B, T, dtype=torch.float64, device="cuda")
    grad = torch.zeros(B, T, V, dtype=torch.float64, device="cuda") if case["grad"] else None
    for b in range(B):
        z = st["logits"][b].double()
        logq = torch.log_softmax(z / tau, dim=-1)
        p = torch.zeros_like(z)
        t = st["teacher"][b].double() / tau
        t[st["idx"][b] < 0] = NEG
        p.scatter_add_(1, st["idx"][b].clamp(min=0).long(), torch.softmax(t, dim=-1))
        w = st["weights"][b].double()
        row = (1 - alpha) * tau ** 2 * torch.where(p > 0, p * (torch.log(p) - logq), torch.zeros_like(p)).sum(-1)
        d = (1 - alpha) * tau * (torch.exp(logq) - p)
        if alpha > 0:
            one = torch.log_softmax(z, dim=-1)
            y = st["labels"][b].long()
            row = row - alpha * one[torch.arange(T, device="cuda"), y]
            d = d + alpha * torch.exp(one)
            d[torch.arange(T, device="cuda"), y] -= alpha
        rows[b] = w * row
        if case["grad"]:
            grad[b] = w[:, None] * d
    return (rows.sum(dim=1), grad if case["grad"] else rows)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, st)
    if case["op"] == "attention":
        return _exact_attention(case, st)
    return _exact_distill(case, st)
