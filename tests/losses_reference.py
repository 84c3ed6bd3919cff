"""Plain references of the losses over rows of logits in float64, with bounds of
what float32 arithmetic as documented may lose (units of u = 2^-24).

An exponential is exp2((z - m) c), c = log2(e) / T in float32: the difference,
the product and c (a rounded constant divided) are off by u, u and 1.5 u of
themselves, so the exponent X by 3.5 u X, the exponential by 3.5 ln2 u X + 2 u
of itself (the exponential function: one unit in the last place).  Formed as
fma(z, c, -round(m c)) it is off by 1.5 u X for c and u X for its one rounding;
the rounding of m c is the same for all that is compared with m.  Two or three
such factors meet where parts of a row are joined; X is then the distance from
the largest logit all the same.  A sum of V terms in threads and a tree has a
depth of at most V / 64 + 16 roundings (64 lanes and more hold V / 64 each, then 6
to 14 levels; 16 lanes hold up to V / 16 of rows of up to 512, then 4 levels: 20 at
V = 256, where the first is 20 as well, 36 at 512).  The exponential function
gives 0 below 2^-126, so a probability may be off by 2^-126 besides (the sum is at
least 1)."""
import math

import torch

U, TINY = 2.0 ** -24, 2.0 ** -126


def depth(n):
    return max(n / 64 + 16, min(n, 512) / 16 + 4)


def softmax(x, m=None):
    """(probabilities, their relative error bounds, log2 of the sum, its error):
    x = z / T in float64, rows with at least one finite value."""
    X = (x.amax(1, keepdim=True) - x) / math.log(2)
    e = torch.exp2(-X)
    s = e.sum(1, keepdim=True)
    far = torch.where(e > 0, X, torch.zeros_like(X))
    rel = (3 * 3.5 * math.log(2) * far + 12) * U
    rel_s = (e * rel).sum(1, keepdim=True) / s + depth(x.shape[1]) * U
    return e / s, rel + rel_s + 6 * U, torch.log2(s), rel_s / math.log(2) + 2 * U * torch.log2(s), X


def distill(z, ids, teacher, temperature=1.0, weights=None):
    """(losses, their bounds, gradient, its bounds before the rounding to the
    result's type).  Rows that have an answer only."""
    z, t, ids = z.double(), teacher.double(), ids.long()
    T = torch.tensor(float(temperature), dtype=torch.float32).double().item()
    n, V = z.shape
    w = torch.ones(n, dtype=torch.float64, device=z.device) if weights is None else weights.double()
    there = (ids >= 0) & (t > -math.inf)
    some = there.any(1)
    q, dq, ls, es, Xs = softmax(z / T)
    t = torch.where(there, t, -math.inf)
    t[~some] = 0.0
    p, dp, lt, et, Xt = softmax(t / T)
    p = p * there
    at = ids.clamp(min=0)
    xs, xt = Xs.gather(1, at), torch.where(there, Xt, torch.zeros_like(Xt))
    gap = torch.where(p > 0, -xt - lt + xs + ls, torch.zeros_like(p))
    xs = torch.where(p > 0, xs, torch.zeros_like(xs))
    losses = T * T * math.log(2) * (p * gap).sum(1)
    k = ids.shape[1]
    err = U * (7 * (xt + xs) + 5 * (lt + ls)) + et + es + gap.abs() * (dp + (depth(k) + 8) * U)
    bound = 1.1 * T * T * math.log(2) * (p * err).sum(1) + 4 * U * losses.abs()
    mass = torch.zeros_like(q).scatter_add_(1, at, p)
    lost = torch.zeros_like(q).scatter_add_(1, at, p * (dp + 8 * U))
    by = (w * T)[:, None] * some[:, None]
    grad = by * (q - mass)
    return losses, bound, grad, 1.1 * by.abs() * (q * (dq + 4 * U) + lost + TINY) + 4 * U * grad.abs()


def balance(z, ids, weight=1.0):
    """(loss, bound, counts, gradient, bounds)."""
    z, ids = z.double(), ids.long()
    if ids.dim() == 1:
        ids = ids[:, None]
    n, K = z.shape
    counted = (ids >= 0).any(1)
    counts = torch.bincount(ids[ids >= 0].flatten(), minlength=K)
    C, R = int(counts.sum()), int(counted.sum())
    scale = K / (C * R) if C else 0.0
    c = counts.double()[None, :]
    p, dp, _, _, _ = softmax(torch.where(counted[:, None], z, 0.0))
    p = p * counted[:, None]
    d = (p * c).sum(1, keepdim=True)
    err = (p * c * dp).sum(1, keepdim=True) + (depth(K) + 8) * U * d
    loss = scale * d.sum()
    grad = weight * scale * p * (c - d)
    bounds = 1.1 * abs(weight) * scale * ((c - d).abs() * (p * (dp + 8 * U) + TINY) + p * (err + 2 * U * (c + d)))
    return loss, 1.1 * scale * err.sum() + 4 * U * loss, counts, grad, bounds
