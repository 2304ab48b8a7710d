"""The sequence operators by their definitions, in 64 bits and with explicit masks (test oracle)."""
import math

import torch


def rotary(x, table, positions, interleaved=False, inverse=False):
    """x [B, T, H, D], table fp64 or fp32 [P, R], positions [B, T]."""
    R = table.shape[1]
    row = table.double()[positions.long()]
    c, s = row[..., :R // 2].unsqueeze(2), row[..., R // 2:].unsqueeze(2)
    s = -s if inverse else s
    y = x.double().clone()
    a = slice(0, R, 2) if interleaved else slice(0, R // 2)
    b = slice(1, R, 2) if interleaved else slice(R // 2, R)
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def table(R, P, theta=10000.0, scaling="plain", factor=1.0, context=4096.0, slow=1.0, fast=32.0):
    out = torch.empty(P, R, dtype=torch.float64)
    for j in range(R // 2):
        f, mag = theta ** (-2.0 * j / R), 1.0
        if scaling == "base" and R > 2:
            f = (theta * factor ** (R / (R - 2))) ** (-2.0 * j / R)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            g = min(max((context * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
            f, mag = f * ((1 - g) / factor + g), 0.1 * math.log(factor) + 1.0
        angle = torch.arange(P, dtype=torch.float64) * f
        out[:, j], out[:, R // 2 + j] = torch.cos(angle) * mag, torch.sin(angle) * mag
    return out


def visible(T, S, lq, lk, causal, window):
    """Truth values [T, S]: which keys each query of one example sees."""
    see = torch.zeros(T, S, dtype=torch.bool)
    for t in range(lq):
        last = t + lk - lq
        lo, hi = 0, lk - 1
        if causal:
            hi = min(hi, last)
        if window:
            lo = max(lo, last - window + 1)
        if hi >= lo:
            see[t, lo:hi + 1] = True
    return see


U = 2.0 ** -24     # unit roundoff of fp32
ETA = 2.0 ** -126  # what is below it may be flushed to 0 (also by bf16, whose range is fp32's)


def attention(q, k, v, causal=False, window=0, scale=None, q_lens=None, k_lens=None, do=None, r=0.0):
    """(o, lse) or, with do, (o, lse, dq, dk, dv), each a pair (value in fp64, error bound).

    The bounds are componentwise and first order, for a computation that keeps scores,
    statistics, differences and sums in fp32 (unit roundoff U; a sum of n products is off by
    at most n U times the sum of their sizes) and rounds the probabilities, their
    gradients and the outputs to a type of unit roundoff r (0: fp32):
      scores         es = (D + 4) U scale sum |q||k|
      lse, P         E  = 2 max es + (n + 16) U + 8 U max |S|, relative for P
      o              sum P|v| (E + r + n U) + (r + U)|o|
      delta          sum |do| (error of o) + (D + 4) U sum |do||o|      (o as it was stored)
      dS             P (|dP - delta| (E + 4 U) + (D + 4) U sum |do||v| + error of delta) + r |dS|
      dq, dk, dv     the same sums over the errors of dS and P, + n U and r of the result.
    Every probability, gradient of one and result may also lose ETA to underflow.
    Where a query sees one key its P is 1 and its dS cancels to 0: no bound relative to the
    result could hold there."""
    B, T, Hq, D = q.shape
    S, Hk = k.shape[1], k.shape[2]
    scale = scale or 1.0 / math.sqrt(D)
    z = dict(dtype=torch.float64, device=q.device)
    shapes = dict(o=(B, T, Hq, D), lse=(B, Hq, T), dq=(B, T, Hq, D), dk=(B, S, Hk, D), dv=(B, S, Hk, D))
    val = {n: torch.zeros(x, **z) for n, x in shapes.items()}
    err = {n: torch.zeros(x, **z) for n, x in shapes.items()}
    val["lse"].fill_(-math.inf)
    c = (D + 4) * U
    for b in range(B):
        lq = T if q_lens is None else max(0, min(T, int(q_lens[b])))
        lk = S if k_lens is None else max(0, min(S, int(k_lens[b])))
        see = visible(T, S, lq, lk, causal, window).to(q.device)
        rows, keys = see.any(1), see.any(0)
        if not bool(rows.any()):
            continue
        see = see[rows][:, keys]
        n, nt = see.sum(1, keepdim=True), T * (Hq // Hk)
        for h in range(Hq):
            g = h // (Hq // Hk)
            Q, K, V = q[b, rows, h].double(), k[b, keys, g].double(), v[b, keys, g].double()
            s = Q @ K.T * scale
            es = torch.where(see, c * scale * (Q.abs() @ K.abs().T), 0.0)
            top = torch.where(see, s.abs(), 0.0).amax(1, keepdim=True)
            E = 2 * es.amax(1, keepdim=True) + (n + 16) * U + 8 * U * top
            s = s.masked_fill(~see, -math.inf)
            y = torch.logsumexp(s, 1)
            p = torch.exp(s - y[:, None])
            O = p @ V
            eO = (p @ V.abs()) * (E + r + n * U) + (r + U) * O.abs() + ETA * (see.double() @ V.abs() + 1)
            val["o"][b, rows, h], err["o"][b, rows, h] = O, eO
            val["lse"][b, h, rows], err["lse"][b, h, rows] = y, E[:, 0] + 4 * U * y.abs()
            if do is None:
                continue
            G = do[b, rows, h].double()
            x = G @ V.T - (G * O).sum(1, keepdim=True)
            edel = (G.abs() * eO).sum(1, keepdim=True) + c * (G.abs() * O.abs()).sum(1, keepdim=True)
            dS = p * x
            eS = p * (x.abs() * (E + 4 * U) + c * (G.abs() @ V.abs().T) + edel) + r * dS.abs()
            eS = eS + ETA * (x.abs() + 1) * see
            eP = p * (E + r + nt * U) + ETA * see
            val["dq"][b, rows, h] = dS @ K * scale
            err["dq"][b, rows, h] = (eS + n * U * dS.abs()) @ K.abs() * scale + (r + 2 * U) * (dS @ K * scale).abs() + ETA
            val["dk"][b, keys, g] += dS.T @ Q * scale
            err["dk"][b, keys, g] += (eS + nt * U * dS.abs()).T @ Q.abs() * scale
            val["dv"][b, keys, g] += p.T @ G
            err["dv"][b, keys, g] += eP.T @ G.abs()
    for m in ("dk", "dv"):
        err[m] += (r + 2 * U) * val[m].abs() + ETA
    return tuple((val[m], err[m]) for m in (("o", "lse") if do is None else ("o", "lse", "dq", "dk", "dv")))


def distill(logits, indices, teacher, labels=None, weights=None, upstream=None, tau=1.0, alpha=0.0):
    """(loss [B], rows [B, T], dlogits [B, T, V]), fp64, row by row."""
    B, T, V = logits.shape
    z64 = dict(dtype=torch.float64, device=logits.device)
    rows, grad = torch.zeros(B, T, **z64), torch.zeros(B, T, V, **z64)
    for b in range(B):
        for t in range(T):
            w = 1.0 if weights is None else float(weights[b, t])
            if w == 0.0:
                continue
            z = logits[b, t].double()
            have = indices[b, t] >= 0
            l, d = torch.zeros((), **z64), torch.zeros(V, **z64)
            if bool(have.any()):
                k = indices[b, t][have].long()
                p = torch.softmax(teacher[b, t][have].double() / tau, 0)
                logq = torch.log_softmax(z / tau, 0)
                pos = p > 0
                l = l + (1 - alpha) * tau ** 2 * (p[pos] * (torch.log(p[pos]) - logq[k[pos]])).sum()
                d = d + (1 - alpha) * tau * torch.exp(logq).index_add(0, k, -p)
            y = -1 if labels is None else int(labels[b, t])
            if y >= 0 and alpha > 0:
                logp = torch.log_softmax(z, 0)
                l = l - alpha * logp[y]
                e = torch.exp(logp)
                e[y] -= 1.0
                d = d + alpha * e
            rows[b, t] = w * l
            grad[b, t] = (1.0 if upstream is None else float(upstream[b])) * w * d
    return rows.sum(1), rows, grad
