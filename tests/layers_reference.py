"""Embeddings, layer norms and log probabilities by their definitions in 64 bits, each value with a bound on the
error of a computation whose sums and statistics are fp32 and whose outputs are rounded once (test oracle).

The bounds are componentwise and first order: U is fp32's unit roundoff, r that of the output's type (0: fp32),
and a sum of terms in a chain of n additions is off by at most n U times the sum of their sizes."""
import torch

U = 2.0 ** -24
ETA = 2.0 ** -126   # what is below it may be flushed to 0
EX2 = 2.0 ** -21    # relative error of the hardware's 2^x, with its argument's last rounding


def layer_norm(x, w=None, b=None, eps=1e-5, dy=None, r=0.0, rw=0.0, per_example=False):
    """x, dy [B, T, D].  (y,) or, with dy, (y, dx, dw, db), each a pair (value, bound); rw: the parameters'
    output rounding."""
    x = x.double()
    B, T, D = x.shape
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(D, dtype=torch.float64, device=x.device) if b is None else b.double()
    c = 48 * U   # a row's sums: at most 32 additions a thread, 10 over threads
    mu = x.mean(-1, keepdim=True)
    emu = c * x.abs().mean(-1, keepdim=True) + U * mu.abs()
    d = x - mu
    var = (d * d).mean(-1, keepdim=True)
    # of the sum of squares, of each difference (its rounding and emu, which cancels to first order)
    evar = (c + 4 * U) * var + emu ** 2 + 2 * U * d.abs().mean(-1, keepdim=True) * emu
    rs = 1.0 / torch.sqrt(var + eps)
    ers = rs * (0.5 * evar / (var + eps) + 6 * U)
    h = d * rs
    eh = rs * (emu + U * d.abs()) + d.abs() * ers + 2 * U * h.abs()
    y = h * w + b
    out = [(y, w.abs() * eh + 2 * U * (w * h).abs() + 2 * U * b.abs() + (r + U) * y.abs() + ETA)]
    if dy is None:
        return tuple(out)
    g = dy.double()
    u = g * w
    s0, s1 = u.mean(-1, keepdim=True), (u * h).mean(-1, keepdim=True)
    e0 = c * u.abs().mean(-1, keepdim=True)
    e1 = (u.abs() * eh).mean(-1, keepdim=True) + c * (u * h).abs().mean(-1, keepdim=True)
    t = u - s0 - h * s1
    dx = rs * t
    et = e0 + h.abs() * e1 + eh * s1.abs() + 4 * U * (u.abs() + s0.abs() + (h * s1).abs())
    out.append((dx, rs * et + ers * t.abs() + (r + 2 * U) * dx.abs() + ETA))
    dims = 1 if per_example else (0, 1)
    n = (T if per_example else B * T) + 20
    dw, db = (g * h).sum(dims), g.sum(dims)
    out.append((dw, (g.abs() * eh).sum(dims) + n * U * (g * h).abs().sum(dims) + rw * dw.abs() + ETA))
    out.append((db, n * U * g.abs().sum(dims) + rw * db.abs() + ETA))
    return tuple(out)


def embedding(tokens, w, scale=1.0, r=0.0):
    y = w.double()[tokens.long()] * scale
    return y, (r + U) * y.abs() + ETA


def embedding_grad(tokens, dy, V, scale=1.0, padding=None, factors=None, r=0.0):
    """((dw, bound), (sqnorms, bound)) of tokens [B, T] and dy [B, T, D]."""
    B, T = tokens.shape
    D = dy.shape[2]
    z = dict(dtype=torch.float64, device=dy.device)
    dw, size, sq, esq = torch.zeros(V, D, **z), torch.zeros(V, D, **z), torch.zeros(B, **z), torch.zeros(B, **z)
    count = torch.zeros(V, 1, **z)
    for i in range(B):
        keep = (tokens[i] >= 0) & (tokens[i] < V)
        if padding is not None:
            keep &= tokens[i] != padding
        t, g = tokens[i][keep].long(), dy[i][keep].double() * scale
        n = torch.zeros(V, 1, **z).index_add_(0, t, torch.ones(len(t), 1, **z))
        one, mag = torch.zeros(V, D, **z).index_add_(0, t, g), torch.zeros(V, D, **z).index_add_(0, t, g.abs())
        sq[i] = (one * one).sum()
        # of the runs' sums; then squares and sums over columns, slabs and positions
        esq[i] = 2 * (one.abs() * mag * (n + 2) * U).sum() + (T / 32 + D / 256 + 64) * U * sq[i] + ETA
        f = 1.0 if factors is None else float(factors[i])
        dw += f * one
        size += abs(f) * mag
        count += n
    return (dw, (count + 4) * U * size + r * dw.abs() + ETA), (sq, esq)


def logprobs(logits, tokens, tau=1.0, dl=None, dh=None, r=0.0, threads=128):
    """Pairs (logprob, entropy, log p) or with dl and dh (logprob, entropy, log p, dz); tokens [B, T], < 0: none."""
    z = logits.double()
    V = z.shape[-1]
    m = z.amax(-1, keepdim=True)
    x = (z - m) / tau
    ls = torch.log(torch.exp(x).sum(-1, keepdim=True))
    lp = x - ls
    p = torch.exp(lp)
    px = torch.where(p > 0, p * x.abs(), torch.zeros_like(p))
    chain = (V / (2 * threads) + 64) * U   # a thread's additions (two chains), and those over threads and parts
    term = EX2 * p + 4 * U * px  # of each e^x: of 2^x, and of x
    es = term.sum(-1, keepdim=True) + chain
    els = es + 2 * U * ls.abs() + U
    elp = 4 * U * x.abs() + els + 2 * U * lp.abs()
    hval = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1, keepdim=True)
    eh = els + torch.where(p > 0, x.abs() * term, torch.zeros_like(p)).sum(-1, keepdim=True) + \
        px.sum(-1, keepdim=True) * (es + chain + 8 * U) + 4 * U * (ls.abs() + hval.abs())
    y = tokens.clamp(min=0).long().unsqueeze(-1)
    given = tokens >= 0
    one, eone = torch.gather(lp, 2, y).squeeze(-1), torch.gather(elp, 2, y).squeeze(-1)
    out = [(torch.where(given, one, 0.0), torch.where(given, eone, 0.0)), (hval.squeeze(-1), eh.squeeze(-1)), (lp, elp)]
    if dl is None and dh is None:
        return tuple(out)
    l = (torch.where(given, dl.double(), 0.0) if dl is not None else torch.zeros_like(one)).unsqueeze(-1)
    k = (dh.double() if dh is not None else torch.zeros_like(one)).unsqueeze(-1)
    inner = -l - k * (torch.where(p > 0, lp, torch.zeros_like(lp)) + hval)
    dz = p * inner
    dz = dz.scatter_add(2, y, torch.where(given.unsqueeze(-1), l, 0.0)) / tau
    ep = EX2 + 4 * U * x.abs() + els + 2 * U * ls.abs()
    ein = k.abs() * (eh + els) + 6 * U * (l.abs() + k.abs() * (hval + ls.abs() + x.abs()))
    err = torch.where(p > 0, p * (ep * inner.abs() + ein), torch.zeros_like(p)) + (ETA + 2.0 ** -149) * (1 + inner.abs())
    err = torch.where(torch.isfinite(err), err, torch.zeros_like(err)) / tau + (r + 3 * U) * dz.abs() + \
        2 * U * l.abs() / tau * torch.zeros_like(p).scatter_(2, y, 1.0) + ETA
    out.append((dz, err))
    return tuple(out)


def top(logits, K):
    """Indices of the K largest logits, of equal ones the lower index first."""
    return torch.sort(logits.double(), dim=-1, descending=True, stable=True)[1][..., :K]
