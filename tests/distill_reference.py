"""A head's distillation loss and its gradients in 64 bits, with bounds of what 32-bit arithmetic and the
roundings to 16 bits may add (as in tests/ops_reference.py).

Bounds.  y = scale t is rounded in units of log 2 (2^-23 of it, twice: the factor and the product), the
teacher's level the same; exp2 and log2 are off by a unit each (2^-23 relative, and 2^-23 of the
logarithm): log q is off by 2^-21 (|y| + |L|) + 2^-20, q relative by as much and 2^-20 more."""
import math

import torch

from tests import ops_reference as ref


def teacher(gen, m, n, top, kind="mixed", extra=3):
    """(index, logit) as m x top views of wider rows on the GPU; what is behind the rows would be far off.
    mixed: different columns, some entries and some whole rows that do not count, one logit of -inf."""
    index = torch.full((m, top + extra), 5, dtype=torch.int64)
    logit = torch.full((m, top + extra), 1e30)
    for r in range(m):
        index[r, :top] = torch.randperm(n, generator=gen)[:top] if top <= n else torch.randint(0, n, (top,), generator=gen)
    logit[:, :top] = torch.randn(m, top, generator=gen) * 3 + 4
    if kind == "mixed":
        index[1::3, top // 2:top] = torch.tensor([-1, n, -100, n + 7])[torch.arange(top - top // 2) % 4]
        index[2::5, :top] = -1
        logit[3::4, 0] = -math.inf
        logit[4::7, :top] = -math.inf
    if kind == "twice" and top > 1:
        index[:, top - 1] = index[:, 0]
        index[::2, top // 2] = index[::2, 0]
    return index.cuda()[:, :top], logit.cuda()[:, :top]


def shares64(index, logit, n, scale, lse):
    """(q, its relative error, log q, error of log q, who counts)."""
    index, logit = index.cpu(), logit.double().cpu()
    counts = (index >= 0) & (index < n)
    y = torch.where(counts, logit * scale, torch.full_like(logit, -math.inf))
    level = torch.logsumexp(y, 1) if lse is None else lse.double().cpu()
    log_q = torch.where(y == -math.inf, y, y - level[:, None])
    q = log_q.exp()
    size = torch.where(y == -math.inf, torch.zeros_like(y), y.abs()) + torch.where(level.abs() < 1e30, level.abs(), torch.zeros_like(level))[:, None]
    log_err = 2.0 ** -21 * size + 2.0 ** -20
    return q, log_err + 2.0 ** -20, log_q, log_err, counts & (y > -math.inf)


def distill64(x, w, index, logit, scale, lse_t, alpha, k):
    """A dict of loss, lse and picked with their bounds, and what the gradient takes further."""
    z, z_err = ref.product64(x, w.t(), k, alpha)
    m, n = z.shape
    lse = torch.logsumexp(z, 1)
    lse_err = z_err.max(1).values + 2.0 ** -18 + 2.0 ** -21 * lse.abs()
    q, q_err, log_q, log_err, has = shares64(index, logit, n, scale, lse_t)
    column = (index.cpu() >= 0) & (index.cpu() < n)
    at = torch.where(column, index.cpu(), torch.zeros_like(index.cpu()))
    picked = torch.where(column, z.gather(1, at), torch.zeros_like(q))
    # (FP32 sums of k products, by lanes: at most k roundings)
    picked_err = torch.where(column, z_err.gather(1, at) + (k + 8) * 2.0 ** -24 * (abs(alpha) * (x.double().cpu().abs() @ w.double().cpu().abs().t())).gather(1, at), torch.zeros_like(q))
    gap = torch.where(has, torch.where(has, log_q, torch.zeros_like(log_q)) - picked + lse[:, None], torch.zeros_like(q))
    terms = q * gap
    size = torch.where(has, torch.where(has, log_q, torch.zeros_like(log_q)).abs() + picked.abs() + lse.abs()[:, None], torch.zeros_like(q))
    err = q * (log_err + picked_err + lse_err[:, None] + 2.0 ** -22 * size) + q_err * terms.abs()
    err = torch.where(has, err, torch.zeros_like(err))
    loss_err = err.sum(1) + (q.shape[1] + 8) * 2.0 ** -24 * (q * size).sum(1)
    return dict(loss=terms.sum(1), loss_err=loss_err, lse=lse, lse_err=lse_err, picked=picked, picked_err=picked_err, z=z, z_err=z_err,
                q=q, q_err=q_err, at=at, has=has)


def distill_grad64(x, w, d, grad, alpha, k, t):
    """(dX, bound, dW, bound) from distill64's dict, P rounded to the type for the products."""
    z, q = d["z"], torch.where(d["has"], d["q"], torch.zeros_like(d["q"]))
    m, n = z.shape
    mass = q.sum(1)
    mass_err = (q * d["q_err"]).sum(1) + 2.0 ** -22 * mass
    p = torch.exp(z - d["lse"][:, None])
    first = p * mass[:, None]
    p_err = first * (d["z_err"] + d["lse_err"][:, None] + 2.0 ** -17) + p * mass_err[:, None]
    at = d["at"]
    # at the teacher's columns the logit is the picked one
    p_err.scatter_add_(1, at, torch.where(d["has"], q * d["q_err"] + first.gather(1, at) * d["picked_err"], torch.zeros_like(q)))
    first = first.scatter_add(1, at, -q)
    counts = mass > 0
    weight = torch.where(counts, grad.double().cpu(), torch.zeros(m, dtype=torch.float64))
    first = torch.where(counts[:, None], first * weight[:, None], torch.zeros_like(first))
    p_err = torch.where(counts[:, None], p_err * weight.abs()[:, None], torch.zeros_like(first))
    # the rounding; FP16's weights are brought to 2^13 first (see tests/ops_reference.py)
    most = float((weight.abs() * mass.clamp(min=1.0)).max()) if m else 0.0
    step = 2.0 ** -38 * most if t == "f16" else 0.0
    p_err = p_err + torch.finfo(ref.TYPES[t]).eps / 2 * (first.abs() + p_err) + step + 2.0 ** -22 * first.abs()
    p_err = torch.where(counts[:, None], p_err, torch.zeros_like(p_err))
    xd, wd = x.double().cpu(), w.double().cpu()
    xd = torch.where(counts[:, None], xd, torch.zeros_like(xd))   # nothing of the others' rows
    dx, dw = alpha * (first @ wd), alpha * (first.t() @ xd)
    dx_err = abs(alpha) * (p_err @ wd.abs()) + ref.sum_error(n + 256, abs(alpha) * (first.abs() @ wd.abs())) + 2.0 ** -22 * dx.abs()
    dw_err = abs(alpha) * (p_err.t() @ xd.abs()) + ref.sum_error(m, abs(alpha) * (first.abs().t() @ xd.abs())) + 2.0 ** -22 * dw.abs()
    return dx, dx_err + ref.rounding(dx, t), dw, dw_err + ref.rounding(dw, t)
