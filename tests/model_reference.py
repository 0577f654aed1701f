"""Plain references of the model's operators (include/vrc_model.h) in 64 bits, from
their definitions, with bounds of what an evaluation in fp32 may be off by.  They share
no code with the HIP path.

The bounds are first order: U is half a step of fp32, and a sum of values whose
longest chain of additions is D is off by at most D U times the sum of magnitudes."""
from __future__ import annotations

import torch

U = 2.0**-24
EPS_HALF = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}     # half a step, relative
TINY_HALF = {torch.float32: 2.0**-150, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}  # half a step of the subnormals


def spans(count, n):
    """The ranks' runs of `count` rows: equal ones, the last with the remainder."""
    each = count // n
    return [(c * each, (c + 1) * each if c < n - 1 else count) for c in range(n)]


def rounded(y, tol, dtype):
    """The bound of y's evaluation, rounded to a type."""
    return tol + (y.abs() + tol) * EPS_HALF[dtype] + TINY_HALF[dtype]


def parts_of(send, join):
    """Lists of sources, one list for each part."""
    if join == "each":
        return [[x] for x in send]
    if join == "sum":
        return [send]
    return [[x[a:b] for x in send] for a, b in spans(send[0].shape[0], len(send))]


def fold(xs):
    """The sum of a part's sources and its bound."""
    xs = [x.double() for x in xs]
    total = torch.stack(xs).sum(0)
    return total, len(xs) * U * torch.stack(xs).abs().sum(0)


def depth(width):
    """Additions that a row's sum chains at most: a lane's elements (33, or one of each
    1024 of a wide row), six across a wave, sixteen across waves, and the product with
    1 / width."""
    return 64 + width / 1024


def layer_norm(xs, residual, weight, bias, eps, center):
    """(y, h, mean, rstd) of one part's sources, and their bounds."""
    h, eh = fold(xs + ([] if residual is None else [residual]))
    w, b = weight.double(), torch.zeros_like(weight.double()) if bias is None else bias.double()
    width = h.shape[-1]
    d = depth(width)
    mean = h.mean(-1, keepdim=True) if center else torch.zeros_like(h[..., :1])
    emean = (eh.mean(-1, keepdim=True) + (d + 2) * U * h.abs().mean(-1, keepdim=True)) if center else torch.zeros_like(mean)
    off = h - mean
    eoff = eh + emean + U * off.abs()
    var = off.square().mean(-1, keepdim=True)
    evar = (2 * off.abs() * eoff + eoff.square()).mean(-1, keepdim=True) + (d + 3) * U * var
    rstd = (var + eps).rsqrt()
    rel = 0.5 * evar / (var + eps) + 4 * U
    x = off * rstd
    y = x * w + b
    ey = w.abs() * (eoff * rstd + x.abs() * (rel + 2 * U)) + U * (y.abs() + b.abs()) + (x * w).abs() * rel * rel
    return (y, ey), (h, eh), (mean[..., 0], emean[..., 0]), (rstd[..., 0], (rstd * rel)[..., 0])


def layer_norm_grad(dys, h, weight, mean, rstd, dh):
    """((dx, bound), (sum of dy x, bound), (sum of dy, bound)) of one part."""
    dy, edy = fold(dys)
    w, width = weight.double(), dy.shape[-1]
    d = depth(width)
    center = mean is not None
    r = rstd.double().unsqueeze(-1)
    x = (h.double() - (mean.double().unsqueeze(-1) if center else 0.0)) * r
    ex = 2 * U * x.abs()
    g = dy * w
    eg = edy * w.abs() + U * g.abs()
    level = g.mean(-1, keepdim=True) if center else torch.zeros_like(r)
    elevel = eg.mean(-1, keepdim=True) + (d + 2) * U * g.abs().mean(-1, keepdim=True) if center else torch.zeros_like(r)
    along = (g * x).mean(-1, keepdim=True)
    ealong = (eg * x.abs() + g.abs() * ex).mean(-1, keepdim=True) + (d + 2) * U * (g * x).abs().mean(-1, keepdim=True)
    dx = r * (g - level - x * along)
    edx = r * (eg + elevel + U * (g - level).abs() + ex * along.abs() + x.abs() * ealong + 2 * U * (x * along).abs()
               + U * (g - level - x * along).abs()) + 2 * U * dx.abs()
    if dh is not None:
        dx = dx + dh.double()
        edx = edx + U * dx.abs()
    rows = dy.reshape(-1, width).shape[0]
    t, et = (dy * x).reshape(-1, width), (edy * x.abs() + dy.abs() * ex + U * (dy * x).abs()).reshape(-1, width)
    s, es = dy.reshape(-1, width), edy.reshape(-1, width)
    return ((dx, edx), (t.sum(0), et.sum(0) + (rows + 32) * U * t.abs().sum(0)),
            (s.sum(0), es.sum(0) + (rows + 32) * U * s.abs().sum(0)))


def logits(hidden, weight):
    """z over the whole vocabulary, and its bound."""
    h, w = hidden.double().reshape(-1, hidden.shape[-1]), torch.cat([x.double() for x in weight])
    return h @ w.t(), (h.shape[-1] + 1) * U * (h.abs() @ w.abs().t())


def cross_entropy(hidden, weight, target, ignore):
    """((loss, bound), (lse, bound)) for finite logits."""
    z, ez = logits(hidden, weight)
    vocab = z.shape[1]
    lse = torch.logsumexp(z, 1)
    # the sum's chain, the exponentials' own error, and their argument's rounding, which
    # is largest relative to the sum where |x| exp(x) is (x = z - max, at most 1 / e of a step each)
    spread = (z.max(1).values - z.min(1).values)
    elsum = (128 + vocab / 2048) * U + 4 * U * (1 + spread.clamp(max=100.0))
    elsecond = ez.max(1).values
    elat = elsecond + elsum + 4 * U * (lse.abs() + z.max(1).values.abs())
    t = target.reshape(-1)
    ok = (t >= 0) & (t < vocab)
    at = t.clamp(0, vocab - 1).unsqueeze(1)
    loss = lse - z.gather(1, at)[:, 0]
    eloss = elat + ez.gather(1, at)[:, 0] + U * loss.abs()
    loss = torch.where(ok, loss, torch.full_like(loss, float("nan")))
    loss = torch.where(t == ignore, torch.zeros_like(loss), loss)
    return (loss, eloss), (lse, elat)


def cross_entropy_grad(hidden, weight, target, lse, dloss, dlse, ignore, dtype):
    """((dhidden, bound), [(dweight, bound) per rank]); the gradients of the logits are
    rounded to `dtype` on the way."""
    z, ez = logits(hidden, weight)
    t, vocab = target.reshape(-1), z.shape[1]
    kept = t != ignore
    b = torch.where(kept, dloss.double().reshape(-1), torch.zeros_like(z[:, 0]))
    a = b + (dlse.double().reshape(-1) if dlse is not None else 0.0)
    live = ((a != 0) | (b != 0)).unsqueeze(1)
    h = torch.where(live, hidden.double().reshape(z.shape[0], -1), torch.zeros((), dtype=torch.float64, device=z.device))
    w = torch.cat([x.double() for x in weight])
    off = z - lse.double().reshape(-1, 1)
    p = torch.where(live, off.exp() * a.unsqueeze(1), torch.zeros_like(z))
    ep = torch.where(live, p.abs() * (ez + 4 * U * (1 + off.abs()) + 2 * U), torch.zeros_like(z))
    g = p.clone()
    rows = torch.nonzero(kept & (t >= 0) & (t < vocab))[:, 0]
    g[rows, t[rows]] -= b[rows]
    eg = ep + 4 * U * (p.abs() + g.abs())
    most = max(float(a.abs().max()), float(b.abs().max())) if a.numel() else 0.0
    if dtype is not torch.float32:
        eg = eg + (g.abs() + eg) * EPS_HALF[dtype]
        if dtype is torch.float16:
            eg = eg + torch.where(live, torch.full_like(g, 2.0**-25 * most * 2.0**-14), torch.zeros_like(g))
    dh, edh = g @ w, eg @ w.abs() + (vocab + 160) * U * (g.abs() @ w.abs())
    dw, edw = g.t() @ h, eg.t() @ h.abs() + (z.shape[0] + 4) * U * (g.abs().t() @ h.abs())
    out, at = [], 0
    for x in weight:
        out.append((dw[at:at + x.shape[0]], edw[at:at + x.shape[0]]))
        at += x.shape[0]
    return (dh, edh), out
